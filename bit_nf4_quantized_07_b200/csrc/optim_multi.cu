// One AdamW update over a list of tensors, with 32-bit or 8-bit states: the
// optimizer step of many LoRA factors in one call.
//
// Pages: deck "3 QLoRA Finetuning" cards 1 and 5 (only the adapters are
// updated; paged optimizer states); "LoRA 与 QLoRA" QLoRA usage notes (the
// paged AdamW of the adapter parameters).  The update is the published AdamW
// (Loshchilov & Hutter, "Decoupled Weight Decay Regularization", ICLR 2019),
// decay first:
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;  p = p (1 - lr wd);
//   p = p - (lr / (1 - b1^t)) m / (sqrt(v / (1 - b2^t)) + eps)
//
// 8-bit states.  Blocks of 256 consecutive elements of a tensor share one fp32
// scale b = max|x| / 448 (formed as max|x| times fp32(1/448)) and hold the E4M3
// codes of fp32(x / b), the group format that the double quantization uses for
// the block constants.  The first moment is held as x = m, the second as
// x = sqrt(v): its square spans 2^36 within a block instead of 2^18.  A nonzero
// sqrt(v) is never rounded to zero (it takes the smallest code): a zero
// denominator under a nonzero m would turn the step into lr m / eps.  The update
// itself runs in fp32 on the restored states, and uses the new v before it is
// rounded.  Per element its 18 bytes leave about 100 issue slots at the HBM rate:
// with correctly rounded quotients and roots throughout, the step needed all of
// them (448 tensors, 40 M elements: 226 us, 49 % of the HBM rate).  So the step
// takes the hardware's approximate root and quotient (2 and 4 units of 2^-24),
// and the codes come from a product with 1 / b; where a value lies so near to the
// middle between two codes that those errors could decide (in one warp of a
// hundred), the warp forms its roots and quotients again, correctly rounded.  A
// code is a sixteenth of its value: one that fell the other way by an error of
// 2^-23 would be seen in the steps after it.
//
// 448 tensors, 40 M elements with BF16 copies take 209 us (5.7 TB/s) with 32-bit
// states, HBM-bound, and 157 us (4.6 TB/s) with 8-bit ones: there 75
// instructions per element fill 56 % of the issue slots, a warp waits for its
// loads 37 % of the time, and the four warps of a scheduler overlap the two only
// in part.  The tensors' pointers travel as a kernel
// parameter (up to 32 KB), so nothing is copied or allocated and a captured
// launch holds its own table.  A tensor is cut into chunks of 2048 elements;
// CTA i takes an equal contiguous share of all chunks, finds its first tensor
// by bisection and walks on from there.
#include "qln_common.cuh"
#include "qln_internal.h"

namespace qln {

constexpr int kMtChunk = 2048;   // elements per CTA step: 256 threads x 8
constexpr int kMtThreads = 256;
constexpr int kMtCtas = 4;       // per SM, one wave
constexpr int kBlock8 = QLN_ADAMW8_BLOCK;
constexpr float kE4m3Max = 448.f;

// Tensors per launch: the table and its arguments stay within the 32,764
// bytes of a launch's parameters.  Short lists take a short table (the launch
// copies all of it: 14 tensors 6.0 us a call instead of 7.1).
constexpr int kMtMax = 480, kMtFew = 48;
struct MtArgs {
    float lr, b1, b2, eps, wd;
    const int64_t *step;
    int count;
};
template <typename Tensor, int N>
struct MtTable {
    MtArgs a;
    uint32_t chunk0[N + 1];  // first chunk of each tensor; [count] = all chunks
    Tensor t[N];
};
static_assert(sizeof(MtTable<qln_adamw_tensor, kMtMax>) <= 32764 && sizeof(MtTable<qln_adamw8_tensor, kMtMax>) <= 32764,
              "kernel parameter limit");

// b^t by squaring (t >= 1), binary64: relative error about t 2^-53 while b^t
// is not negligible against 1.
__device__ __forceinline__ double pow_int(double b, int64_t t) {
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) r *= b;
        b *= b;
        if (b == 0.0 && t > 1) return 0.0;
    }
    return r;
}

struct MtStep {
    float step_size, inv_sqrt_bc2;
};

// The step's two factors, formed by one thread of the CTA.
__device__ __forceinline__ MtStep mt_step(const MtArgs &a) {
    const int64_t tv = *a.step;
    const int64_t t = tv < 1 ? 1 : tv;  // a step below 1 is taken as the first
    MtStep s;
    s.step_size = (float)((double)a.lr / (1.0 - pow_int((double)a.b1, t)));
    s.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - pow_int((double)a.b2, t)));
    return s;
}

// One element in fp32.
__device__ __forceinline__ void mt_elem(float &p, float g, float &m, float &v, const MtArgs &a, const MtStep &s) {
    m = __fadd_rn(__fmul_rn(a.b1, m), __fmul_rn(1.0f - a.b1, g));
    v = __fadd_rn(__fmul_rn(a.b2, v), __fmul_rn(1.0f - a.b2, __fmul_rn(g, g)));
    p = __fmul_rn(p, 1.0f - a.lr * a.wd);
    const float denom = __fadd_rn(__fmul_rn(__fsqrt_rn(v), s.inv_sqrt_bc2), a.eps);
    p = __fsub_rn(p, __fmul_rn(s.step_size, __fdiv_rn(m, denom)));
}

// The CTA's share of the chunks and the tensor its first chunk lies in.
struct MtRange {
    uint32_t c, end;
    int ti;
};
template <typename Table>
__device__ __forceinline__ MtRange mt_range(const Table &T) {
    const uint64_t total = T.chunk0[T.a.count];
    MtRange r;
    r.c = (uint32_t)(total * blockIdx.x / gridDim.x);
    r.end = (uint32_t)(total * (blockIdx.x + 1) / gridDim.x);
    int lo = 0, hi = T.a.count;  // chunk0[lo] <= c < chunk0[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (T.chunk0[mid] <= r.c) lo = mid;
        else hi = mid;
    }
    r.ti = lo;
    return r;
}

template <int N>
__global__ void __launch_bounds__(kMtThreads, kMtCtas)
adamw_multi_kernel(const __grid_constant__ MtTable<qln_adamw_tensor, N> T) {
    __shared__ MtStep sh;
    MtRange R = mt_range(T);
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0) sh = mt_step(T.a);
    __syncthreads();
    const MtStep S = sh;
    for (; R.c < R.end; ++R.c) {
        while (R.c >= T.chunk0[R.ti + 1]) ++R.ti;
        const qln_adamw_tensor &t = T.t[R.ti];
        const int64_t e0 = (int64_t)(R.c - T.chunk0[R.ti]) * kMtChunk;
        const int64_t left = t.n - e0;
        if (left >= kMtChunk) {
            float4 p[2], g[2], m[2], v[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t i = (e0 >> 2) + u * kMtThreads + threadIdx.x;
                g[u] = __ldcs(reinterpret_cast<const float4 *>(t.grad) + i);
                m[u] = reinterpret_cast<const float4 *>(t.m)[i];
                v[u] = reinterpret_cast<const float4 *>(t.v)[i];
                p[u] = reinterpret_cast<const float4 *>(t.param)[i];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t i = (e0 >> 2) + u * kMtThreads + threadIdx.x;
                mt_elem(p[u].x, g[u].x, m[u].x, v[u].x, T.a, S);
                mt_elem(p[u].y, g[u].y, m[u].y, v[u].y, T.a, S);
                mt_elem(p[u].z, g[u].z, m[u].z, v[u].z, T.a, S);
                mt_elem(p[u].w, g[u].w, m[u].w, v[u].w, T.a, S);
                reinterpret_cast<float4 *>(t.param)[i] = p[u];
                reinterpret_cast<float4 *>(t.m)[i] = m[u];
                reinterpret_cast<float4 *>(t.v)[i] = v[u];
                if (t.param_bf16)
                    reinterpret_cast<uint2 *>(t.param_bf16)[i] =
                        make_uint2(pack_bf16x2(p[u].x, p[u].y), pack_bf16x2(p[u].z, p[u].w));
            }
        } else {  // a tensor's last chunk: element by element
            for (int64_t i = e0 + threadIdx.x; i < t.n; i += kMtThreads) {
                float p = t.param[i], m = t.m[i], v = t.v[i];
                mt_elem(p, t.grad[i], m, v, T.a, S);
                t.param[i] = p;
                t.m[i] = m;
                t.v[i] = v;
                if (t.param_bf16) t.param_bf16[i] = __bfloat16_as_ushort(__float2bfloat16_rn(p));
            }
        }
    }
}

// ---- 8-bit states ------------------------------------------------------------
// Four codes of one word -> fp32, times the block's scale.
__device__ __forceinline__ void e4m3x4_restore(uint32_t w, float b, float *x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w >> (16 * h)) & 0xffffu), __NV_E4M3);
        const float2 f = __half22float2(__half2(r));
        x[2 * h] = __fmul_rn(f.x, b);
        x[2 * h + 1] = __fmul_rn(f.y, b);
    }
}
// Four values already divided by the scale -> codes (round to nearest even;
// NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x4_pack(const float *y) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
// sqrt(x) within 2 units of 2^-24.
__device__ __forceinline__ float root_approx(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// One element; v: the restored root of v on entry, the new v on return.
__device__ __forceinline__ void mt_elem8(float &p, float g, float &m, float &v, const MtArgs &a, const MtStep &s,
                                         float decay) {
    m = __fmaf_rn(1.0f - a.b1, g, __fmul_rn(a.b1, m));
    v = __fmaf_rn(1.0f - a.b2, __fmul_rn(g, g), __fmul_rn(a.b2, __fmul_rn(v, v)));
    const float denom = __fmaf_rn(root_approx(v), s.inv_sqrt_bc2, a.eps);
    p = __fmaf_rn(-s.step_size, __fdividef(m, denom), __fmul_rn(p, decay));
}
constexpr uint32_t kInfBits = 0x7f800000u;
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// A block's scale b, and 1 / b (0 if b is 0; infinite if b is below about 2^-128).
__device__ __forceinline__ void block_scale(float top, float &inv, float &b) {
    b = __fmul_rn(top, 1.0f / kE4m3Max);
    inv = b > 0.f ? __frcp_rn(b) : 0.f;
}
constexpr float kLess = 1.f - 0x1p-20f, kMore = 1.f + 0x1p-20f;
__device__ __forceinline__ float least_root(float v) { return v > 0.f ? 0.001953125f : 0.f; }  // 2^-9, the smallest code

// The codes of four elements by their definition; rarely called, and a call, so that it takes no registers of the others.
__device__ __noinline__ uint2 codes_exact(float4 m, float4 v, float bm, float bv) {
    const float x[8] = {m.x, m.y, m.z, m.w, v.x, v.y, v.z, v.w};
    float y[4], z[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        y[k] = bm > 0.f ? __fdiv_rn(x[k], bm) : 0.f;
        z[k] = fmaxf(bv > 0.f ? __fdiv_rn(__fsqrt_rn(x[4 + k]), bv) : 0.f, least_root(x[4 + k]));
    }
    return make_uint2(e4m3x4_pack(y), e4m3x4_pack(z));
}

// A warp takes one block per step and requests the next two ones' 2.5 KB each
// before it works on the present one's; a tensor's partial last block is read in
// its turn.  448 tensors, 40 M elements: 157 us with two CTAs per SM; 162 us with
// three and one block ahead, whose 80 registers spill.
constexpr int k8Ctas = 2;

template <int N>
__global__ void __launch_bounds__(kMtThreads, k8Ctas)
adamw8_multi_kernel(const __grid_constant__ MtTable<qln_adamw8_tensor, N> T) {
    static_assert(kBlock8 == 256 && kMtChunk == 8 * kBlock8, "one block per warp and step");
    __shared__ MtStep sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    MtRange R = mt_range(T);
    pdl_wait();
    pdl_trigger();
    struct Raw {  // this lane's 8 elements of a whole block
        float4 g[2], p[2];
        uint2 m, v;
        float bm, bv;
    };
    Raw n1, n2;
    uint32_t ac = R.c;  // the look-ahead: its chunk and tensor
    int ati = R.ti;
    auto request = [&](Raw &nxt) {
        if (ac < R.end) {
            while (ac >= T.chunk0[ati + 1]) ++ati;
            const qln_adamw8_tensor &t = T.t[ati];
            const int64_t blk = (int64_t)(ac - T.chunk0[ati]) * (kMtChunk / kBlock8) + warp;
            if ((blk + 1) * kBlock8 <= t.n) {
                const int64_t e = blk * kBlock8 + 8 * lane;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    nxt.g[h] = __ldcs(reinterpret_cast<const float4 *>(t.grad + e) + h);
                    nxt.p[h] = *(reinterpret_cast<const float4 *>(t.param + e) + h);
                }
                nxt.m = *reinterpret_cast<const uint2 *>(t.m + e);
                nxt.v = *reinterpret_cast<const uint2 *>(t.v + e);
                nxt.bm = t.m_scale[blk];
                nxt.bv = t.v_scale[blk];
            }
        }
        ++ac;
    };
    request(n1);
    request(n2);
    if (threadIdx.x == 0) sh = mt_step(T.a);
    __syncthreads();
    const MtStep S = sh;
    const float decay = 1.0f - T.a.lr * T.a.wd;
    for (; R.c < R.end; ++R.c) {
        const Raw cur = n1;
        n1 = n2;
        request(n2);
        while (R.c >= T.chunk0[R.ti + 1]) ++R.ti;
        const qln_adamw8_tensor &t = T.t[R.ti];
        const int64_t blk = (int64_t)(R.c - T.chunk0[R.ti]) * (kMtChunk / kBlock8) + warp;
        const int64_t e = blk * kBlock8 + 8 * lane;  // this lane's 8 elements
        if (blk * kBlock8 >= t.n) continue;
        const bool whole = (blk + 1) * kBlock8 <= t.n;
        const int64_t left = t.n - e;
        float p[8], g[8], m[8], v[8];
        if (whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                g[4 * h] = cur.g[h].x, g[4 * h + 1] = cur.g[h].y, g[4 * h + 2] = cur.g[h].z, g[4 * h + 3] = cur.g[h].w;
                p[4 * h] = cur.p[h].x, p[4 * h + 1] = cur.p[h].y, p[4 * h + 2] = cur.p[h].z, p[4 * h + 3] = cur.p[h].w;
            }
            e4m3x4_restore(cur.m.x, cur.bm, m);
            e4m3x4_restore(cur.m.y, cur.bm, m + 4);
            e4m3x4_restore(cur.v.x, cur.bv, v);
            e4m3x4_restore(cur.v.y, cur.bv, v + 4);
        } else {
            const float bm = t.m_scale[blk], bv = t.v_scale[blk];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const bool in = k < left;
                g[k] = in ? t.grad[e + k] : 0.f;
                p[k] = in ? t.param[e + k] : 0.f;
                m[k] = in ? __fmul_rn(e4m3_to_f32(t.m[e + k]), bm) : 0.f;
                v[k] = in ? __fmul_rn(e4m3_to_f32(t.v[e + k]), bv) : 0.f;
            }
        }
        uint32_t am = 0, av = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            mt_elem8(p[k], g[k], m[k], v[k], T.a, S, decay);
            am = max(am, abs_bits(m[k]));
            av = max(av, abs_bits(v[k]));
        }
        if (whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *(reinterpret_cast<float4 *>(t.param + e) + h) = make_float4(p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]);
            if (t.param_bf16)
                *reinterpret_cast<uint4 *>(t.param_bf16 + e) =
                    make_uint4(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]), pack_bf16x2(p[6], p[7]));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < left) {
                    t.param[e + k] = p[k];
                    if (t.param_bf16) t.param_bf16[e + k] = __bfloat16_as_ushort(__float2bfloat16_rn(p[k]));
                }
        }
        am = __reduce_max_sync(0xffffffffu, am);
        av = __reduce_max_sync(0xffffffffu, av);
        const bool odd = max(am, av) >= kInfBits;  // an element is not finite: it sets no scale and becomes NaN
        if (odd) {
            am = av = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                am = max(am, abs_bits(m[k]) < kInfBits ? abs_bits(m[k]) : 0u);
                av = max(av, abs_bits(v[k]) < kInfBits ? abs_bits(v[k]) : 0u);
            }
            am = __reduce_max_sync(0xffffffffu, am);
            av = __reduce_max_sync(0xffffffffu, av);
        }
        float im, iv, nm, nv;
        block_scale(__uint_as_float(am), im, nm);
        block_scale(__fsqrt_rn(__uint_as_float(av)), iv, nv);  // the largest root: the root is monotone
        // The codes of values 2^-20 smaller and 2^-20 larger: the errors of the root, of 1 / b and of the products (at
        // most 5 units of 2^-24) lie within, so where both agree the value between them has that code.
        const float im0 = __fmul_rn(im, kLess), im1 = __fmul_rn(im, kMore), iv0 = __fmul_rn(iv, kLess), iv1 = __fmul_rn(iv, kMore);
        uint32_t mo[2], vo[2], diff = __float_as_uint(fmaxf(im1, iv1)) >= kInfBits;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float y0[4], y1[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y0[k] = __fmul_rn(m[4 * h + k], im0);
                y1[k] = __fmul_rn(m[4 * h + k], im1);
            }
            mo[h] = e4m3x4_pack(y0);
            diff |= mo[h] ^ e4m3x4_pack(y1);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float x = root_approx(v[4 * h + k]), lo = least_root(v[4 * h + k]);
                y0[k] = fmaxf(__fmul_rn(x, iv0), lo);
                y1[k] = fmaxf(__fmul_rn(x, iv1), lo);
            }
            vo[h] = e4m3x4_pack(y0);
            diff |= vo[h] ^ e4m3x4_pack(y1);
        }
        if (__any_sync(0xffffffffu, diff != 0)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2 c = codes_exact(make_float4(m[4 * h], m[4 * h + 1], m[4 * h + 2], m[4 * h + 3]),
                                            make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]), nm, nv);
                mo[h] = c.x;
                vo[h] = c.y;
            }
        }
        if (odd) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (abs_bits(m[k]) >= kInfBits) mo[k / 4] |= 0x7fu << (8 * (k % 4));
                if (abs_bits(v[k]) >= kInfBits) vo[k / 4] |= 0x7fu << (8 * (k % 4));
            }
        }
        __syncwarp();  // every lane has read the scales
        if (lane == 0) {
            t.m_scale[blk] = nm;
            t.v_scale[blk] = nv;
        }
        if (whole) {
            *reinterpret_cast<uint2 *>(t.m + e) = make_uint2(mo[0], mo[1]);
            *reinterpret_cast<uint2 *>(t.v + e) = make_uint2(vo[0], vo[1]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < left) {
                    t.m[e + k] = (uint8_t)(mo[k / 4] >> (8 * (k % 4)));
                    t.v[e + k] = (uint8_t)(vo[k / 4] >> (8 * (k % 4)));
                }
        }
    }
}

// ---- host ----------------------------------------------------------------------
static cudaError_t page_tensor(const qln_adamw_tensor &t, bool in, int dev, cudaStream_t st) {
    const size_t b = (size_t)t.n * 4;
    cudaError_t e;
    if (in && ((e = page_managed(t.param, b, dev, st)) != cudaSuccess || (e = page_managed(t.grad, b, dev, st)) != cudaSuccess)) return e;
    if ((e = page_managed(t.m, b, dev, st)) != cudaSuccess) return e;
    return page_managed(t.v, b, dev, st);
}
static cudaError_t page_tensor(const qln_adamw8_tensor &t, bool in, int dev, cudaStream_t st) {
    const size_t b = (size_t)t.n, s = (size_t)((t.n + kBlock8 - 1) / kBlock8) * 4;
    cudaError_t e;
    if (in && ((e = page_managed(t.param, 4 * b, dev, st)) != cudaSuccess || (e = page_managed(t.grad, 4 * b, dev, st)) != cudaSuccess)) return e;
    if ((e = page_managed(t.m, b, dev, st)) != cudaSuccess || (e = page_managed(t.v, b, dev, st)) != cudaSuccess) return e;
    if ((e = page_managed(t.m_scale, s, dev, st)) != cudaSuccess) return e;
    return page_managed(t.v_scale, s, dev, st);
}

// The update itself, N tensors at a time at most.
template <typename Tensor, int N>
static cudaError_t launch_tables(void (*kernel)(const MtTable<Tensor, N>), int ctas, const Tensor *tensors, int count,
                                 const MtArgs &args, cudaStream_t st, int num_sms) {
    MtTable<Tensor, N> T;
    T.a = args;
    for (int i0 = 0; i0 < count; i0 += T.a.count) {
        const int k = count - i0 < N ? count - i0 : N;
        uint64_t chunks = 0;
        T.a.count = k;
        for (int i = 0; i < k; ++i) {
            T.chunk0[i] = (uint32_t)chunks;
            T.t[i] = tensors[i0 + i];
            chunks += (uint64_t)(tensors[i0 + i].n + kMtChunk - 1) / kMtChunk;
        }
        T.chunk0[k] = (uint32_t)chunks;
        const uint64_t wave = (uint64_t)num_sms * ctas;
        const cudaError_t e = launch_pdl(kernel, dim3((unsigned)(chunks < wave ? chunks : wave)), dim3(kMtThreads), 0, st, T);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename Tensor>
static cudaError_t launch_multi(void (*few)(const MtTable<Tensor, kMtFew>), void (*many)(const MtTable<Tensor, kMtMax>),
                                int ctas, const Tensor *tensors, int count, const qln_adamw_config *cfg,
                                const int64_t *step, int flags, cudaStream_t st, int num_sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (flags & QLN_ADAMW_PAGE_IN)
        for (int i = 0; i < count; ++i)
            if ((e = page_tensor(tensors[i], true, dev, st)) != cudaSuccess) return e;
    const MtArgs a{cfg->lr, cfg->beta1, cfg->beta2, cfg->eps, cfg->weight_decay, step, 0};
    e = count <= kMtFew ? launch_tables(few, ctas, tensors, count, a, st, num_sms)
                        : launch_tables(many, ctas, tensors, count, a, st, num_sms);
    if (e != cudaSuccess) return e;
    if (flags & QLN_ADAMW_PAGE_OUT)
        for (int i = 0; i < count; ++i)
            if ((e = page_tensor(tensors[i], false, cudaCpuDeviceId, st)) != cudaSuccess) return e;
    return cudaSuccess;
}

cudaError_t launch_adamw_multi(const qln_adamw_tensor *t, int count, const qln_adamw_config *cfg, const int64_t *step,
                               int flags, cudaStream_t st, int num_sms) {
    return launch_multi<qln_adamw_tensor>(adamw_multi_kernel<kMtFew>, adamw_multi_kernel<kMtMax>, kMtCtas, t, count, cfg, step, flags, st, num_sms);
}
cudaError_t launch_adamw8_multi(const qln_adamw8_tensor *t, int count, const qln_adamw_config *cfg, const int64_t *step,
                                int flags, cudaStream_t st, int num_sms) {
    return launch_multi<qln_adamw8_tensor>(adamw8_multi_kernel<kMtFew>, adamw8_multi_kernel<kMtMax>, k8Ctas, t, count, cfg, step, flags, st, num_sms);
}

}  // namespace qln

// Residual sum with RMSNorm, an E4M3 output, and the backward.
//
//   s = x + res                      stored rounded to the model dtype
//   r = 1 / sqrt(mean(s^2) + eps)    of the unrounded fp32 sum
//   y = g * s * r                    model dtype
//   c = max |y| / 448, q = E4M3(y / c)   one scale per row
// and, with sh = s * r, t = g * dy:
//   dx = dsum + r * (t - sh * mean(t * sh)),   dg = sum over rows of dy * sh
//
// Bound by the bytes of the rows: a row is read once, stays in registers
// between the two reductions (sum of squares, largest |y|) and is written
// once.  A CTA of `tpr` threads holds a row, CPT 16-byte chunks per thread.
// Forward of 32768 x 2560 bf16 with both outputs: 140 us, 5.4 TB/s of its 755
// MB; backward of 16381 x 2560: 64 us, 5.2 TB/s.
#include <algorithm>

#include <cuda_fp8.h>

#include "ctx.cuh"
#include "tc.cuh"

namespace engram {
namespace {

constexpr int kMaxCpt = 8;
constexpr int kMaxTpr = 512;       // threads per row at most
constexpr float kE4M3Max = 448.f;

struct NormGeo {
    int cpt, tpr, rb;   // chunks per thread, threads per row (whole warps), rows per CTA (tpr == 32 only)
};

// `cpt` chunks per thread (one in the forward, two in the backward, which keeps
// a running sum per column) while the row fits kMaxTpr threads, more for wider
// rows; rows of at most a warp's share go eight to a CTA.  False above
// kMaxTpr * kMaxCpt chunks.  Forward of 32768 x 2560 bf16 with both outputs:
// 140 us with one, two or (144 us) five chunks, 213 us with a warp per row;
// of 256 rows 3.1, 3.7, 5.8 and 9.8 us.
bool norm_geo(int cpr, int cpt, NormGeo& g) {
    g.cpt = cpt;
    while (g.cpt < kMaxCpt && cpr > kMaxTpr * g.cpt) g.cpt <<= 1;
    g.tpr = ((cpr + g.cpt - 1) / g.cpt + 31) / 32 * 32;
    g.rb = g.tpr == 32 ? 8 : 1;
    return g.tpr <= kMaxTpr;
}

// |f| as ordered bits: NaN above infinity, so a maximum keeps it
__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the row's threads: the warps' sums in warp order.  `slot` differs
// between uses within a row, so one barrier serves each.
__device__ __forceinline__ float row_sum(float v, float* slot, int warps, int warp, int lane) {
    v = warp_sum(v);
    if (warps == 1) return v;
    if (lane == 0) slot[warp] = v;
    __syncthreads();
    float t = lane < warps ? slot[lane] : 0.f;
    return warp_sum(t);
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* slot, int warps, int warp, int lane) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (warps == 1) return v;
    if (lane == 0) slot[warp] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < warps ? slot[lane] : 0u);
}

template <int N>
__device__ __forceinline__ void store_e4m3(uint8_t* to, const float* f) {
    uint32_t w[N / 4];
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k], f[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k + 2], f[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
        w[k] = a | (b << 16);
    }
    if constexpr (N == 8) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(to) = w[0];
}

// ---------------------------------------------------------------- forward

template <typename T, int CPT>
__global__ void __launch_bounds__(kMaxTpr) add_norm_kernel(const T* x, const T* res, int64_t n, int cpr, const float* __restrict__ gain, float eps,
                                T* sum_out, T* y, uint8_t* q, float* q_scale, float* rstd) {
    constexpr int EPC = Vec<T>::N;
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= n) return;                       // whole warps: rows per CTA only with one warp per row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int64_t base = row * cpr;
    float f[CPT][EPC];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = tid + k * blockDim.x;
        if (c < cpr) {
            Vec<T>::load(x + (base + c) * EPC, f[k]);
        } else {
#pragma unroll
            for (int j = 0; j < EPC; ++j) f[k][j] = 0.f;
        }
    }
    if (res) {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = tid + k * blockDim.x;
            if (c < cpr) {
                float a[EPC];
                Vec<T>::load(res + (base + c) * EPC, a);
#pragma unroll
                for (int j = 0; j < EPC; ++j) f[k][j] += a[j];
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = tid + k * blockDim.x;
        if (sum_out && c < cpr) Vec<T>::store(sum_out + (base + c) * EPC, f[k]);
#pragma unroll
        for (int j = 0; j < EPC; ++j) ss = fmaf(f[k][j], f[k][j], ss);
    }
    ss = row_sum(ss, s_sum, warps, warp, lane);
    const float r = rsqrtf(ss / (float)(cpr * EPC) + eps);
    if (rstd && tid == 0) rstd[row] = r;
    if (!y && !q) return;
    // p = g * s; y = p * r, and the codes y / c = 448 p / max |p| without r, so that a code's value has
    // three roundings behind it
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = tid + k * blockDim.x;
        if (c < cpr) {
            if (gain) {
#pragma unroll
                for (int j = 0; j < EPC; j += 4) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(gain + c * EPC + j));
                    f[k][j] *= v.x; f[k][j + 1] *= v.y; f[k][j + 2] *= v.z; f[k][j + 3] *= v.w;
                }
            }
            float o[EPC];
#pragma unroll
            for (int j = 0; j < EPC; ++j) {
                o[j] = f[k][j] * r;
                amax = max(amax, abs_bits(f[k][j]));
            }
            if (y) Vec<T>::store(y + (base + c) * EPC, o);
        }
    }
    if (!q) return;
    const float top = __uint_as_float(row_max(amax, s_max, warps, warp, lane));
    if (tid == 0) q_scale[row] = top * r / kE4M3Max;
    // one reciprocal per row; a row whose reciprocal would overflow divides instead, and a row of zeros
    // (scale 0) has codes 0
    const bool tiny = top < 1e-35f;
    const float inv = kE4M3Max / top;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = tid + k * blockDim.x;
        if (c < cpr) {
            float o[EPC];
#pragma unroll
            for (int j = 0; j < EPC; ++j) o[j] = tiny ? (top > 0.f ? f[k][j] / top * kE4M3Max : 0.f) : f[k][j] * inv;
            store_e4m3<EPC>(q + (base + c) * EPC, o);
        }
    }
}

// ---------------------------------------------------------------- backward

// Rows blockIdx.x, blockIdx.x + gridDim.x, ... (times rb); each thread keeps
// the running sums of dg for its columns and writes them once per CTA row.
template <typename T, int CPT>
__global__ void __launch_bounds__(kMaxTpr) add_norm_grad_kernel(const T* d_y, const T* d_sum, const T* __restrict__ sum,
                                     const float* __restrict__ rstd, int64_t n, int cpr,
                                     const float* __restrict__ gain, T* d_x, float* __restrict__ part) {
    constexpr int EPC = Vec<T>::N;
    __shared__ float s_dot[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    float dg[CPT][EPC];
#pragma unroll
    for (int k = 0; k < CPT; ++k)
#pragma unroll
        for (int j = 0; j < EPC; ++j) dg[k][j] = 0.f;
    const int64_t row0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, step = (int64_t)gridDim.x * blockDim.y;
    // the next row's operands are in flight while a row is worked on
    uint4 qy[CPT], qs[CPT], qd[CPT];
    float r_next = 0.f;
    auto fetch = [&](int64_t row) {
        if (row >= n) return;
        r_next = __ldg(rstd + row);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = tid + k * blockDim.x;
            if (c < cpr) {
                qy[k] = *(reinterpret_cast<const uint4*>(d_y) + row * cpr + c);
                qs[k] = __ldg(reinterpret_cast<const uint4*>(sum) + row * cpr + c);
                if (d_sum) qd[k] = *(reinterpret_cast<const uint4*>(d_sum) + row * cpr + c);
            }
        }
    };
    fetch(row0);
    int flip = 0;
    for (int64_t row = row0; row < n; row += step, flip ^= 1) {
        const int64_t base = row * cpr;
        const float r = r_next;
        float t[CPT][EPC], sh[CPT][EPC], o[CPT][EPC];
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = tid + k * blockDim.x;
            if (c < cpr) {
                Vec<T>::load(reinterpret_cast<const T*>(&qy[k]), t[k]);
                Vec<T>::load(reinterpret_cast<const T*>(&qs[k]), sh[k]);
                if (d_sum) Vec<T>::load(reinterpret_cast<const T*>(&qd[k]), o[k]);
#pragma unroll
                for (int j = 0; j < EPC; ++j) {
                    sh[k][j] *= r;
                    dg[k][j] = fmaf(t[k][j], sh[k][j], dg[k][j]);
                }
                if (gain) {
#pragma unroll
                    for (int j = 0; j < EPC; j += 4) {
                        const float4 v = __ldg(reinterpret_cast<const float4*>(gain + c * EPC + j));
                        t[k][j] *= v.x; t[k][j + 1] *= v.y; t[k][j + 2] *= v.z; t[k][j + 3] *= v.w;
                    }
                }
#pragma unroll
                for (int j = 0; j < EPC; ++j) dot = fmaf(t[k][j], sh[k][j], dot);
            }
        }
        fetch(row + step);
        dot = row_sum(dot, s_dot[flip], warps, warp, lane) / (float)(cpr * EPC);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = tid + k * blockDim.x;
            if (c < cpr) {
#pragma unroll
                for (int j = 0; j < EPC; ++j) {
                    const float v = r * (t[k][j] - sh[k][j] * dot);
                    o[k][j] = d_sum ? o[k][j] + v : v;
                }
                Vec<T>::store(d_x + (base + c) * EPC, o[k]);
            }
        }
    }
    if (!part) return;
    float* to = part + row0 * (int64_t)(cpr * EPC);
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = tid + k * blockDim.x;
        if (c < cpr) {
#pragma unroll
            for (int j = 0; j < EPC; j += 4)
                *reinterpret_cast<float4*>(to + c * EPC + j) = make_float4(dg[k][j], dg[k][j + 1], dg[k][j + 2], dg[k][j + 3]);
        }
    }
}

// dg: 32 columns per CTA, its warps over the partial rows, added in warp order
constexpr int kGainWarps = 32;
__global__ void __launch_bounds__(kGainWarps * 32) gain_grad_kernel(const float* part, int rows, int d, float* d_gain) {
    __shared__ float s_sum[kGainWarps][32];
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float acc = 0.f;
    if (col < d) {
#pragma unroll 8
        for (int r = warp; r < rows; r += kGainWarps) acc += part[(int64_t)r * d + col];
    }
    s_sum[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && col < d) {
        for (int w = 1; w < kGainWarps; ++w) acc += s_sum[w][lane];
        d_gain[col] = acc;
    }
}

// ---------------------------------------------------------------- host side

// CTAs of the backward: each leaves one partial row (times rb) of dg.  One wave
// of what the registers hold, 512 threads an SM (16381 x 2560 bf16: 64 us with
// three CTAs an SM, 68 to 73 us with six to twelve, 102 us before the next
// row's operands were kept in flight).
int64_t grad_ctas(const engram_ctx* c, int64_t n, const NormGeo& g) {
    const int per_sm = std::max(1, 512 / (g.tpr * g.rb));
    return std::max<int64_t>(1, std::min<int64_t>((n + g.rb - 1) / g.rb, (int64_t)c->num_sms * per_sm));
}

template <typename T>
cudaError_t launch_norm(const NormGeo& g, const void* x, const void* res, int64_t n, int d, const float* gain, float eps,
                        void* sum, void* y, void* q, float* q_scale, float* rstd, cudaStream_t s) {
    const int cpr = d / Vec<T>::N;
    const dim3 block(g.tpr, g.rb);
    const unsigned grid = (unsigned)((n + g.rb - 1) / g.rb);
    auto go = [&](auto kern) {
        kern<<<grid, block, 0, s>>>(static_cast<const T*>(x), static_cast<const T*>(res), n, cpr, gain, eps,
                                    static_cast<T*>(sum), static_cast<T*>(y), static_cast<uint8_t*>(q), q_scale, rstd);
    };
    if (g.cpt == 1) go(add_norm_kernel<T, 1>);
    else if (g.cpt == 2) go(add_norm_kernel<T, 2>);
    else if (g.cpt == 4) go(add_norm_kernel<T, 4>);
    else go(add_norm_kernel<T, 8>);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_norm_grad(const engram_ctx* c, const NormGeo& g, const void* d_y, const void* d_sum, const void* sum,
                             const float* rstd, int64_t n, int d, const float* gain, void* d_x, float* part,
                             cudaStream_t s) {
    const int cpr = d / Vec<T>::N;
    const dim3 block(g.tpr, g.rb);
    const unsigned grid = (unsigned)grad_ctas(c, n, g);
    auto go = [&](auto kern) {
        kern<<<grid, block, 0, s>>>(static_cast<const T*>(d_y), static_cast<const T*>(d_sum),
                                    static_cast<const T*>(sum), rstd, n, cpr, gain, static_cast<T*>(d_x), part);
    };
    if (g.cpt == 2) go(add_norm_grad_kernel<T, 2>);
    else if (g.cpt == 4) go(add_norm_grad_kernel<T, 4>);
    else go(add_norm_grad_kernel<T, 8>);
    return cudaGetLastError();
}

engram_status norm_shape(const engram_ctx* c, int64_t n, int cpt, NormGeo& g) {
    if (!c) return inval("null context");
    if (n < 0 || n >= (int64_t)1 << 31) return inval("the row count must be in [0, 2^31)");
    if (!norm_geo(c->cfg.hidden / (16 / c->hs), cpt, g)) {
        set_error("the norm takes hidden widths of at most 32768 (bf16) or 16384 (fp32)");
        return ENGRAM_E_UNSUPPORTED;
    }
    return ENGRAM_OK;
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" {

engram_status engram_add_norm(engram_ctx* c, const void* x, const void* res, int64_t n, const float* gain,
                              void* sum_out, void* y, void* q, float* q_scale, float* rstd, cudaStream_t s) {
    NormGeo g{};
    engram_status st = norm_shape(c, n, 1, g);
    if (st != ENGRAM_OK) return st;
    if (n == 0) return ENGRAM_OK;
    if (!sum_out && !y && !q && !rstd) return inval("no output requested");
    if (!q != !q_scale) return inval("q and q_scale go together");
    if (!x) return inval("null tensor pointer");
    if (!aligned16(x) || !aligned16(res) || !aligned16(gain) || !aligned16(sum_out) || !aligned16(y) || !aligned16(q))
        return inval("x, res, gain, sum_out, y and q must be 16-byte aligned");
    st = check_device(c);
    if (st != ENGRAM_OK) return st;
    prof_reset(c);
    prof_begin(c, s, "add_norm");
    const int d = c->cfg.hidden;
    cudaError_t e = c->hs == 2 ? launch_norm<__nv_bfloat16>(g, x, res, n, d, gain, c->cfg.eps, sum_out, y, q, q_scale, rstd, s)
                               : launch_norm<float>(g, x, res, n, d, gain, c->cfg.eps, sum_out, y, q, q_scale, rstd, s);
    prof_end(c, s);
    return e == cudaSuccess ? ENGRAM_OK : cuda_fail("residual norm launch", e);
}

size_t engram_add_norm_grad_workspace_bytes(const engram_ctx* c, int64_t n) {
    NormGeo g{};
    if (!c || norm_shape(c, n, 2, g) != ENGRAM_OK) return 0;
    return align256((size_t)grad_ctas(c, n, g) * g.rb * c->cfg.hidden * 4);
}

engram_status engram_add_norm_grad(engram_ctx* c, const void* d_y, const void* d_sum, const void* sum, const float* rstd,
                                   int64_t n, const float* gain, void* d_x, float* d_gain, void* workspace,
                                   size_t workspace_bytes, cudaStream_t s) {
    NormGeo g{};
    engram_status st = norm_shape(c, n, 2, g);
    if (st != ENGRAM_OK) return st;
    if (n > 0 && (!d_y || !sum || !rstd || !d_x)) return inval("null tensor pointer");
    if (!aligned16(d_y) || !aligned16(d_sum) || !aligned16(sum) || !aligned16(gain) || !aligned16(d_x))
        return inval("d_y, d_sum, sum, gain and d_x must be 16-byte aligned");
    const size_t need = engram_add_norm_grad_workspace_bytes(c, n);
    if (n > 0 && d_gain) {
        if (!workspace) return inval("null workspace");
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return inval("workspace must be 256-byte aligned");
        if (workspace_bytes < need) {
            set_error("engram_add_norm_grad: the workspace is smaller than engram_add_norm_grad_workspace_bytes");
            return ENGRAM_E_NOMEM;
        }
    }
    st = check_device(c);
    if (st != ENGRAM_OK) return st;
    prof_reset(c);
    const int d = c->cfg.hidden;
    if (n == 0) {
        if (!d_gain) return ENGRAM_OK;
        cudaError_t e = cudaMemsetAsync(d_gain, 0, (size_t)d * 4, s);
        return e == cudaSuccess ? ENGRAM_OK : cuda_fail("clearing the gain gradient", e);
    }
    float* part = d_gain ? static_cast<float*>(workspace) : nullptr;
    prof_begin(c, s, "add_norm_grad");
    cudaError_t e = c->hs == 2 ? launch_norm_grad<__nv_bfloat16>(c, g, d_y, d_sum, sum, rstd, n, d, gain, d_x, part, s)
                               : launch_norm_grad<float>(c, g, d_y, d_sum, sum, rstd, n, d, gain, d_x, part, s);
    prof_end(c, s);
    if (e == cudaSuccess && d_gain) {
        prof_begin(c, s, "gain_grad");
        e = launch_after(c, gain_grad_kernel, (unsigned)((d + 31) / 32), dim3(kGainWarps * 32), 0, s, part,
                         (int)(grad_ctas(c, n, g) * g.rb), d, d_gain);
        prof_end(c, s);
    }
    return e == cudaSuccess ? ENGRAM_OK : cuda_fail("residual norm gradient launches", e);
}

}  // extern "C"

// fp8_quant.cu -- quantisers to 8 bits with a scale for each block of 128, for
// sm_103a: fp8_quantize_rows, _tiles and _columns (include/fp8.h).
//
// All three read each element once and write one byte for it: they are bound by
// memory.  amax is taken over the bit patterns of |x| as integers, which order
// as the numbers do and put NaN above everything, so a NaN reaches its scale.
#include <cstdint>
#include <mutex>

#include <cuda_fp8.h>

#include "../../include/fp8.h"
#include "common.cuh"
#include "fp8.cuh"
#include "ptx.cuh"

namespace dg {
namespace {

constexpr int kBlock = 128;
constexpr int kMaxGroups = 1024;
constexpr int64_t kMaxDim = INT32_MAX - 1024;
constexpr int64_t kMaxLd = int64_t(1) << 38;

template <bool E5M2>
struct Top {
    static constexpr float value = E5M2 ? 57344.0f : 448.0f;
};

// Scale and its reciprocal factor from the bits of a block's amax.
template <bool E5M2>
__device__ __forceinline__ void scale_of(uint32_t amax_bits, float& scale, float& factor) {
    constexpr float top = Top<E5M2>::value;
    const uint32_t least = __float_as_uint(top * 1.17549435e-38f);   // top * 2^-126
    const float amax = __uint_as_float(amax_bits > least ? amax_bits : least);
    scale = __fdiv_rn(amax, top);
    factor = __fdiv_rn(top, amax);
}

template <bool E5M2>
__device__ __forceinline__ uint32_t code2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
}

// Codes of 8 numbers, first in the lowest byte.
template <bool E5M2>
__device__ __forceinline__ uint2 code8(const float (&x)[8], float f) {
    uint2 r;
    r.x = code2<E5M2>(x[0] * f, x[1] * f) | (code2<E5M2>(x[2] * f, x[3] * f) << 16);
    r.y = code2<E5M2>(x[4] * f, x[5] * f) | (code2<E5M2>(x[6] * f, x[7] * f) << 16);
    return r;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Elements [k, k + 8) of a row (zeros at and beyond K).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int64_t k, int64_t K, float (&x)[8]) {
    if (VEC && k + 8 <= K) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = *reinterpret_cast<const float4*>(row + k);
            const float4 b = *reinterpret_cast<const float4*>(row + k + 4);
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
            x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(row + k);
            const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(e[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = k + i < K ? static_cast<float>(row[k + i]) : 0.0f;
    }
}

__device__ __forceinline__ void store8(uint8_t* row, int64_t k, int64_t K, uint2 c) {
    if (k + 8 <= K) {
        *reinterpret_cast<uint2*>(row + k) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < K) row[k + i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

struct QuantParams {
    const void* X;
    int64_t ldx, x_group;
    const int32_t* rows;
    const int32_t* offsets;
    uint8_t* Q;
    int64_t ldq, q_group;
    float* S;
    int64_t s_row, s_blk, s_group;
    int64_t T, R, K;
    int32_t groups;
    int32_t transpose;
};

// ---- rows: 16 lanes per block of 128 (8 elements each), kUnits blocks in flight
// per thread so that enough bytes are outstanding.
constexpr int kUnits = 4;

template <typename T, bool E5M2, bool VEC>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t num_kb = (p.K + kBlock - 1) / kBlock;
    const int64_t total = p.R * num_kb;
    const int l = threadIdx.x & 15;
    const int64_t u0 = int64_t(blockIdx.x) * (16 * kUnits) + (threadIdx.x >> 4);
    float x[kUnits][8];
    int64_t row[kUnits], kb[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int64_t u = u0 + 16 * i;
        row[i] = u / num_kb;
        kb[i] = u - row[i] * num_kb;
        int64_t src = row[i];
        bool there = u < total;
        if (there && p.rows != nullptr) {
            src = p.rows[row[i]];
            there = src >= 0 && src < p.T;
        }
        if (there) {
            load8<T, VEC>(static_cast<const T*>(p.X) + src * p.ldx, kb[i] * kBlock + 8 * l, p.K, x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = umax(m, abs_bits(x[i][e]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = umax(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (u0 + 16 * i >= total) continue;
        float scale, f;
        scale_of<E5M2>(m, scale, f);
        store8(p.Q + row[i] * p.ldq, kb[i] * kBlock + 8 * l, p.K, code8<E5M2>(x[i], f));
        if (l == 0) p.S[row[i] * p.s_row + kb[i] * p.s_blk] = scale;
    }
}

// The codes of a 128 x 128 block, written transposed through shared memory: row
// group rg (8 rows) of column c is 8 bytes at slot rg ^ (c / 8) of column c's 128.
struct Turn {
    uint2 slot[kBlock][16];
};

__device__ __forceinline__ void turn_in(Turn& t, int cg, int rg, const uint2 (&code)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // bytes j of the eight rows' codes
        const uint32_t sel = static_cast<uint32_t>(j & 3);
        uint32_t b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = ((j < 4 ? code[i].x : code[i].y) >> (8 * sel)) & 0xffu;
        t.slot[8 * cg + j][rg ^ cg] =
            make_uint2(b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24),
                       b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24));
    }
}

// Columns of the block as rows of Q: [0, cols) of them, bytes [0, width) at q.
__device__ __forceinline__ void turn_out(const Turn& t, uint8_t* q, int64_t ldq, int cols, int width) {
    for (int u = threadIdx.x; u < kBlock * 16; u += 256) {
        const int c = u >> 4, rg = u & 15;
        if (c < cols && 8 * rg < width) store8(q + c * ldq, 8 * rg, width, t.slot[c][rg ^ (c >> 3)]);
    }
}

// ---- tiles: one 128 x 128 block per CTA; thread = 8 columns of 8 rows.
template <typename T, bool E5M2, bool VEC>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const QuantParams p) {
    __shared__ Turn turn;
    __shared__ uint32_t red[8];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t num_kb = (p.K + kBlock - 1) / kBlock;
    const int64_t num_nb = (p.R + kBlock - 1) / kBlock;
    const int64_t kb = blockIdx.x % num_kb;
    const int64_t nb = (blockIdx.x / num_kb) % num_nb;
    const int64_t g = blockIdx.x / (num_kb * num_nb);
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const T* X = static_cast<const T*>(p.X) + g * p.x_group;
    const int64_t n0 = nb * kBlock, k0 = kb * kBlock;
    float x[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = n0 + 8 * rg + i;
        load8<T, VEC>(X + n * p.ldx, k0 + 8 * cg, n < p.R ? p.K : 0, x[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = umax(m, abs_bits(x[i][e]));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = umax(m, red[w]);
    float scale, f;
    scale_of<E5M2>(m, scale, f);
    uint2 code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) code[i] = code8<E5M2>(x[i], f);
    uint8_t* Q = p.Q + g * p.q_group;
    if (threadIdx.x == 0)
        p.S[g * p.s_group + (p.transpose ? kb * p.s_row + nb * p.s_blk : nb * p.s_row + kb * p.s_blk)] =
            scale;
    const int rows = static_cast<int>(p.R - n0 < kBlock ? p.R - n0 : kBlock);
    const int cols = static_cast<int>(p.K - k0 < kBlock ? p.K - k0 : kBlock);
    if (p.transpose) {
        turn_in(turn, cg, rg, code);
        __syncthreads();
        turn_out(turn, Q + k0 * p.ldq + n0, p.ldq, cols, rows);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (8 * rg + i < rows && 8 * cg < cols)
                store8(Q + (n0 + 8 * rg + i) * p.ldq + k0, 8 * cg, cols, code[i]);
    }
}

// ---- columns: 128 rows of one group x 128 columns per CTA, a scale for each
// column.  blockIdx.x = column tile, blockIdx.y (+ 65535 z) = block of rows.
template <typename T, bool E5M2, bool VEC>
__global__ void __launch_bounds__(256) quantize_columns_kernel(const QuantParams p) {
    __shared__ Turn turn;
    __shared__ uint32_t red[16][kBlock];
    __shared__ int where[2];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t num_ct = (p.K + kBlock - 1) / kBlock;
    const int64_t ct = blockIdx.x % num_ct;
    const int pb = static_cast<int>(blockIdx.x / num_ct);
    // First row of the block and one past its group's last row (equal: no rows).
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int base = 0, lo = 0, hi = 0;
        const int top = static_cast<int>(p.R);
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const int g = g0 + lane;
            int a = 0, b = 0;
            if (g < p.groups) {
                a = p.offsets != nullptr ? p.offsets[g] : 0;
                b = p.offsets != nullptr ? p.offsets[g + 1] : top;
                a = a < 0 ? 0 : (a > top ? top : a);
                b = b < a ? a : (b > top ? top : b);
            }
            const int n = (b - a) / kBlock + ((b - a) % kBlock != 0 ? 1 : 0);
            int sum = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += v;
            }
            const int before = base + sum - n;
            const bool mine = pb >= before && pb < before + n;
            const unsigned who = __ballot_sync(0xffffffffu, mine);
            if (who != 0u) {
                const int src = __ffs(static_cast<int>(who)) - 1;
                lo = __shfl_sync(0xffffffffu, a + (pb - before) * kBlock, src);
                hi = __shfl_sync(0xffffffffu, b, src);
                break;
            }
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) {
            where[0] = lo;
            where[1] = hi;
        }
    }
    __syncthreads();
    const int64_t r0 = where[0], r1 = where[1];
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t c0 = ct * kBlock;
    float x[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        int64_t r = r0 + 8 * rg + i;
        bool there = r < r1;
        if (there && p.rows != nullptr) {
            r = p.rows[r];
            there = r >= 0 && r < p.T;
        }
        load8<T, VEC>(static_cast<const T*>(p.X) + (there ? r : 0) * p.ldx, c0 + 8 * cg,
                      there ? p.K : 0, x[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax(m, abs_bits(x[i][e]));
        red[rg][8 * cg + e] = m;
    }
    __syncthreads();
    if (threadIdx.x < kBlock) {
        const int c = threadIdx.x;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = umax(m, red[i][c]);
        float scale, f;
        scale_of<E5M2>(m, scale, f);
        if (c0 + c < p.K) p.S[(c0 + c) * p.s_row + pb * p.s_blk] = scale;
        red[0][c] = __float_as_uint(f);     // only this thread reads column c of red
    }
    __syncthreads();
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(red[0][8 * cg + e]);
    uint2 code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= f[e];
        code[i] = code8<E5M2>(x[i], 1.0f);
    }
    turn_in(turn, cg, rg, code);
    __syncthreads();
    const int cols = static_cast<int>(p.K - c0 < kBlock ? p.K - c0 : kBlock);
    turn_out(turn, p.Q + c0 * p.ldq + int64_t(pb) * kBlock, p.ldq, cols, kBlock);
}

// ---------------------------------------------------------------- host side

using QuantKernel = void (*)(QuantParams);
enum Kind { kRows, kTiles, kColumns };

template <Kind KIND, typename T, bool E5M2, bool VEC>
QuantKernel kernel_of() {
    if constexpr (KIND == kRows)
        return quantize_rows_kernel<T, E5M2, VEC>;
    else if constexpr (KIND == kTiles)
        return quantize_tiles_kernel<T, E5M2, VEC>;
    else
        return quantize_columns_kernel<T, E5M2, VEC>;
}

template <Kind KIND, typename T>
QuantKernel pick2(bool e5m2, bool vec) {
    if (e5m2) return vec ? kernel_of<KIND, T, true, true>() : kernel_of<KIND, T, true, false>();
    return vec ? kernel_of<KIND, T, false, true>() : kernel_of<KIND, T, false, false>();
}

template <Kind KIND>
QuantKernel pick(int in_type, bool e5m2, bool vec) {
    if (in_type == GEMM_OUT_F32) return pick2<KIND, float>(e5m2, vec);
    if (in_type == GEMM_OUT_F16) return pick2<KIND, __half>(e5m2, vec);
    return pick2<KIND, __nv_bfloat16>(e5m2, vec);
}

std::mutex g_mu;
int g_arch[64] = {};   // 0 unknown, 1 sm_103, 2 another

gemm_status_t device_ok() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    std::lock_guard<std::mutex> lock(g_mu);
    if (g_arch[dev] == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
            (void)cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        g_arch[dev] = major == 10 && minor == 3 ? 1 : 2;
    }
    return g_arch[dev] == 1 ? GEMM_OK : GEMM_ERR_UNSUPPORTED;
}

// Checks that all three share.  x_rows x K elements are read, q_rows x q_cols bytes
// written, for each of `groups` matrices.
gemm_status_t check(const QuantParams& p, int64_t groups, int64_t x_rows, int64_t q_rows,
                    int64_t q_cols, int32_t in_type, int32_t q_type, bool* empty) {
    *empty = true;
    if (p.T < 0 || p.R < 0 || p.K < 0 || groups < 0) return GEMM_ERR_INVALID_ARG;
    if ((in_type != GEMM_OUT_F32 && in_type != GEMM_OUT_F16 && in_type != GEMM_OUT_BF16) ||
        (q_type != FP8_E4M3 && q_type != FP8_E5M2))
        return GEMM_ERR_UNSUPPORTED;
    if (p.T > kMaxDim || p.R > kMaxDim || p.K > kMaxDim || q_cols > kMaxDim) return GEMM_ERR_UNSUPPORTED;
    if (q_rows == 0 || q_cols == 0 || groups == 0) return GEMM_OK;
    *empty = false;
    const int64_t esize = in_type == GEMM_OUT_F32 ? 4 : 2;
    if (p.Q == nullptr || p.S == nullptr || (p.X == nullptr && x_rows > 0 && p.K > 0))
        return GEMM_ERR_INVALID_ARG;
    if (p.ldx < p.K || p.ldq < q_cols || p.ldq % 16 != 0 || p.q_group < 0 || p.q_group % 16 != 0 ||
        p.x_group < 0 || p.s_row < 0 || p.s_blk < 0 || p.s_group < 0)
        return GEMM_ERR_INVALID_ARG;
    if (p.ldx > kMaxLd || p.ldq > kMaxLd || p.x_group > kMaxLd || p.q_group > kMaxLd ||
        p.s_row > kMaxLd || p.s_blk > kMaxLd || p.s_group > kMaxLd)
        return GEMM_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(p.Q) % 16u != 0u || reinterpret_cast<uintptr_t>(p.S) % 4u != 0u ||
        reinterpret_cast<uintptr_t>(p.X) % static_cast<uintptr_t>(esize) != 0u ||
        (reinterpret_cast<uintptr_t>(p.rows) | reinterpret_cast<uintptr_t>(p.offsets)) % 4u != 0u)
        return GEMM_ERR_INVALID_ARG;
    if (groups > 1 && p.q_group < (q_rows - 1) * p.ldq + q_cols) return GEMM_ERR_INVALID_ARG;
    if (x_rows > 0 && p.K > 0) {
        const uintptr_t xl = reinterpret_cast<uintptr_t>(p.X);
        const uintptr_t xh =
            xl + static_cast<uintptr_t>(((groups - 1) * p.x_group + (x_rows - 1) * p.ldx + p.K) * esize);
        const uintptr_t ql = reinterpret_cast<uintptr_t>(p.Q);
        const uintptr_t qh =
            ql + static_cast<uintptr_t>((groups - 1) * p.q_group + (q_rows - 1) * p.ldq + q_cols);
        if (xl < qh && ql < xh) return GEMM_ERR_INVALID_ARG;
    }
    return GEMM_OK;
}

gemm_status_t launch(QuantKernel k, int64_t grid, const QuantParams& p, cudaStream_t stream) {
    if (grid > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
    const gemm_status_t st = device_ok();
    if (st != GEMM_OK) return st;
    if (launch_pdl(k, dim3(static_cast<unsigned>(grid)), dim3(256), size_t(0), stream, p) !=
        cudaSuccess) {
        (void)cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    return GEMM_OK;
}

bool vec_ok(const QuantParams& p, int32_t in_type) {
    const int64_t per16 = in_type == GEMM_OUT_F32 ? 4 : 8;
    return reinterpret_cast<uintptr_t>(p.X) % 16u == 0u && p.ldx % per16 == 0 && p.x_group % per16 == 0;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace
}  // namespace dg

extern "C" {

gemm_status_t fp8_quantize_rows(const void* X, int64_t ldx, int32_t in_type, const int32_t* rows,
                                int64_t T, int64_t R, int64_t K, void* Q, int64_t ldq,
                                int32_t q_type, float* S, int64_t s_row, int64_t s_blk,
                                struct CUstream_st* stream) {
    dg::QuantParams p{};
    p.X = X, p.ldx = ldx, p.rows = rows, p.T = T, p.R = R, p.K = K;
    p.Q = static_cast<uint8_t*>(Q), p.ldq = ldq, p.S = S, p.s_row = s_row, p.s_blk = s_blk;
    bool empty = false;
    const gemm_status_t st =
        dg::check(p, 1, rows != nullptr ? T : R, R, K, in_type, q_type, &empty);
    if (st != GEMM_OK || empty) return st;
    if (rows == nullptr && T < R) return GEMM_ERR_INVALID_ARG;
    const int64_t units = R * dg::cdiv(K, dg::kBlock);
    return dg::launch(dg::pick<dg::kRows>(in_type, q_type == FP8_E5M2, dg::vec_ok(p, in_type)),
                      dg::cdiv(units, 16 * dg::kUnits), p, reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t fp8_quantize_tiles(const void* X, int64_t ldx, int64_t x_group, int32_t in_type,
                                 int64_t groups, int64_t N, int64_t K, int32_t transpose, void* Q,
                                 int64_t ldq, int64_t q_group, int32_t q_type, float* S,
                                 int64_t s_row, int64_t s_blk, int64_t s_group,
                                 struct CUstream_st* stream) {
    dg::QuantParams p{};
    p.X = X, p.ldx = ldx, p.x_group = x_group, p.T = N, p.R = N, p.K = K;
    p.Q = static_cast<uint8_t*>(Q), p.ldq = ldq, p.q_group = q_group;
    p.S = S, p.s_row = s_row, p.s_blk = s_blk, p.s_group = s_group;
    p.transpose = transpose ? 1 : 0;
    bool empty = false;
    const gemm_status_t st = dg::check(p, groups, N, transpose ? K : N, transpose ? N : K, in_type,
                                       q_type, &empty);
    if (st != GEMM_OK || empty) return st;
    return dg::launch(dg::pick<dg::kTiles>(in_type, q_type == FP8_E5M2, dg::vec_ok(p, in_type)),
                      groups * dg::cdiv(N, dg::kBlock) * dg::cdiv(K, dg::kBlock), p,
                      reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t fp8_quantize_columns(const void* X, int64_t ldx, int32_t in_type, const int32_t* rows,
                                   int64_t T, int64_t R, int64_t C, int64_t groups,
                                   const int32_t* offsets, void* Q, int64_t ldq, int32_t q_type,
                                   float* S, int64_t s_row, int64_t s_blk,
                                   struct CUstream_st* stream) {
    if (groups < 0) return GEMM_ERR_INVALID_ARG;
    if (groups > dg::kMaxGroups) return GEMM_ERR_UNSUPPORTED;
    if (groups > 0 && offsets == nullptr) return GEMM_ERR_INVALID_ARG;
    dg::QuantParams p{};
    p.X = X, p.ldx = ldx, p.rows = rows, p.T = T, p.R = R, p.K = C;
    p.groups = static_cast<int32_t>(groups > 0 ? groups : 1);
    p.offsets = groups > 0 ? offsets : nullptr;
    p.Q = static_cast<uint8_t*>(Q), p.ldq = ldq, p.S = S, p.s_row = s_row, p.s_blk = s_blk;
    if (R < 0 || R > dg::kMaxDim) return R < 0 ? GEMM_ERR_INVALID_ARG : GEMM_ERR_UNSUPPORTED;
    const int64_t blocks = R / dg::kBlock + p.groups;
    bool empty = false;
    const gemm_status_t st =
        dg::check(p, 1, rows != nullptr ? T : R, C, blocks * dg::kBlock, in_type, q_type, &empty);
    if (st != GEMM_OK || empty) return st;
    if (rows == nullptr && T < R) return GEMM_ERR_INVALID_ARG;
    return dg::launch(dg::pick<dg::kColumns>(in_type, q_type == FP8_E5M2, dg::vec_ok(p, in_type)),
                      blocks * dg::cdiv(C, dg::kBlock), p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// quantize_transposed.hip -- fp8_quantize_transposed: the block cast of a
// matrix's transpose (and, from the same read, of the matrix itself).
//
// Mathematics: fp8_quantize's, per block of 128 consecutive rows of one
// column (or per 128x128 tile): s = fl32(max(amax, 1e-12) / MAX), codes of
// x / s.  Design: one 256-lane workgroup per 128x128 tile, held in registers,
// every lane with a 16-byte vector of each of RPT consecutive rows.  A
// column's amax is a maximum over the lane's rows, two cross-row exchanges
// and four words of LDS; a row's is four DPP steps over its 16 (32) lanes.
// The transposed codes pass through 16 KiB of LDS: a lane packs its RPT codes
// of a column into one LDS word group, whose place is permuted by the
// column's vector so that the lanes of a row do not all hit one bank, and the
// workgroup then stores whole 128-byte lines of the transposed rows.
#include <hip/hip_runtime.h>

#include "device_fp8.hpp"
#include "gs/training.h"
#include "gs_internal.hpp"

#ifndef GS_MAX_GRID
#define GS_MAX_GRID (1 << 20)
#endif

namespace gsk {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kAmaxFloor = 1e-12f;

template <int FMT>
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    const float a = as_f32(amax_bits);
    return (a > kAmaxFloor ? a : kAmaxFloor) / Fp8<FMT>::kMax;
}

// FP8 codes of four FP32 values (as bits) with one scale from their block's
// amax (so always in div_by_scale's range, and no finite quotient past MAX by
// more than its rounding).  nf: a value may be NaN (-> sign|0x7F) or Inf
// (-> +-MAX).
template <int FMT>
__device__ __forceinline__ uint32_t cast4(const uint32_t (&e)[4], float s, float r, bool nf) {
    constexpr uint32_t kMaxCode = FMT == 0 ? 0x7Eu : 0x7Bu;
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        q[k] = __builtin_copysignf(div_by_scale(__builtin_fabsf(as_f32(e[k])), s, r), as_f32(e[k]));
    uint32_t o = cvt_pk<FMT, true>(q[2], q[3], cvt_pk<FMT, false>(q[0], q[1], 0u));
    if (nf) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((e[k] & 0x7F800000u) == 0x7F800000u) {
                const uint32_t c = ((e[k] >> 24) & 0x80u) | ((e[k] & 0x7FFFFFu) ? 0x7Fu : kMaxCode);
                o = (o & ~(0xFFu << (8 * k))) | (c << (8 * k));
            }
    }
    return o;
}

template <typename IN>
__device__ __forceinline__ uint32_t widen_bits(const IN *p) {
    if constexpr (sizeof(IN) == 2) return uint32_t(*reinterpret_cast<const uint16_t *>(p)) << 16;
    else return *reinterpret_cast<const uint32_t *>(p);
}

struct TransposeArgs {
    int64_t rows, cols, rows_pad;
    int64_t tiles_r, ntiles;
    uint8_t *codes_t, *codes;
    float *scales_t, *scales;
    int32_t *nonfinite;
};

template <int FMT, bool TILE, bool BOTH, typename IN>
__global__ __launch_bounds__(256)
void quant_transposed_kernel(const IN *__restrict__ x, const TransposeArgs p) {
    constexpr int VEC = 16 / int(sizeof(IN));         // columns per lane: 8 or 4
    constexpr int LPR = 128 / VEC;                    // lanes per row: 16 or 32
    constexpr int RPT = 128 / (256 / LPR);            // rows per lane: 8 or 16
    constexpr int UNITS = 128 / RPT;                  // LDS units per column: 16 or 8
    constexpr int WPU = RPT / 4;                      // words per unit: 2 or 4
    __shared__ __align__(16) uint32_t codes_lds[128 * 32];
    __shared__ uint32_t red[4][128];
    const int tid = threadIdx.x;
    const int seg = tid % LPR;                        // which vector of the row
    const int rg = tid / LPR;                         // which group of RPT rows
    bool saw_nf = false;
    for (int64_t t = blockIdx.x; t < p.ntiles; t += gridDim.x) {
        const int64_t tc = t / p.tiles_r, tr = t - tc * p.tiles_r;
        const int64_t row0 = tr * 128 + rg * RPT, col0 = tc * 128 + seg * VEC;
        // widened values, [row][column]
        uint32_t w[RPT][4];                           // the raw vectors
        const bool whole = tr * 128 + 128 <= p.rows && tc * 128 + 128 <= p.cols &&
                           p.cols % VEC == 0;
        if (whole) {
            const IN *src = x + row0 * p.cols + col0;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const u32x4 v = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4 *>(src + i * p.cols));
                w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t word = 0;
#pragma unroll
                    for (int h = 0; h < VEC / 4; ++h) {
                        const int64_t r = row0 + i, c = col0 + q * (VEC / 4) + h;
                        if (r < p.rows && c < p.cols) {
                            const uint32_t b = widen_bits(x + r * p.cols + c);
                            word |= VEC == 8 ? (b >> 16) << (16 * h) : b;
                        }
                    }
                    w[i][q] = word;
                }
        }
        auto elem = [&](int i, int c) -> uint32_t {
            if constexpr (VEC == 8)
                return (c & 1) ? (w[i][c >> 1] & 0xFFFF0000u) : (w[i][c >> 1] << 16);
            else
                return w[i][c];
        };
        // non-finite values are left out of every maximum
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int c = 0; c < VEC; ++c) most = max(most, elem(i, c) & 0x7FFFFFFFu);
        const bool nf = most >= 0x7F800000u;
        saw_nf |= nf;
        auto mag = [&](int i, int c) -> uint32_t {
            const uint32_t a = elem(i, c) & 0x7FFFFFFFu;
            return nf && a >= 0x7F800000u ? 0u : a;
        };
        float cs[VEC];                                // scales of the lane's columns
        float rs[RPT];                                // BOTH: scales of the lane's rows
        if constexpr (TILE) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int c = 0; c < VEC; ++c) m = max(m, mag(i, c));
            m = wave_max(m);
            if ((tid & 63) == 0) red[0][tid >> 6] = m;
            __syncthreads();
            m = max(max(red[0][0], red[0][1]), max(red[0][2], red[0][3]));
            const float s = block_scale<FMT>(m);
#pragma unroll
            for (int c = 0; c < VEC; ++c) cs[c] = s;
            if (tid == 0) {
                p.scales_t[tc * p.tiles_r + tr] = s;
                if (BOTH) p.scales[tr * (p.cols / 128) + tc] = s;
            }
        } else {
            uint32_t cm[VEC];
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < RPT; ++i) m = max(m, mag(i, c));
                if (LPR == 16) m = max(m, (uint32_t)__shfl_xor((int)m, 16));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32));
                cm[c] = m;
            }
            if ((tid & 63) < LPR)
#pragma unroll
                for (int c = 0; c < VEC; ++c) red[tid >> 6][seg * VEC + c] = cm[c];
            __syncthreads();
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const int k = seg * VEC + c;
                cs[c] = block_scale<FMT>(max(max(red[0][k], red[1][k]), max(red[2][k], red[3][k])));
            }
            if (rg == 0)
#pragma unroll
                for (int c = 0; c < VEC; ++c)
                    if (col0 + c < p.cols) p.scales_t[(col0 + c) * p.tiles_r + tr] = cs[c];
        }
        if constexpr (BOTH) {
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                if constexpr (TILE) {
                    rs[i] = cs[0];
                } else {
                    uint32_t m = 0;
#pragma unroll
                    for (int c = 0; c < VEC; ++c) m = max(m, mag(i, c));
                    m = group_max<16>(m);
                    if (LPR == 32) m = max(m, (uint32_t)__shfl_xor((int)m, 16));
                    rs[i] = block_scale<FMT>(m);
                    if (seg == 0 && row0 + i < p.rows)
                        p.scales[(row0 + i) * (p.cols / 128) + tc] = rs[i];
                }
            }
        }
        // transposed codes into LDS
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            const float r = 1.0f / cs[c];
            uint32_t out[WPU];
#pragma unroll
            for (int k = 0; k < WPU; ++k) {
                const uint32_t e[4] = {elem(4 * k, c), elem(4 * k + 1, c), elem(4 * k + 2, c),
                                       elem(4 * k + 3, c)};
                out[k] = cast4<FMT>(e, cs[c], r, nf);
            }
            uint32_t *dst = &codes_lds[(seg * VEC + c) * 32 + (rg ^ (seg & (UNITS - 1))) * WPU];
            if constexpr (WPU == 2) *reinterpret_cast<u32x2 *>(dst) = u32x2{out[0], out[1]};
            else *reinterpret_cast<u32x4 *>(dst) = u32x4{out[0], out[1], out[2], out[3]};
        }
        // row-major codes straight to memory
        if constexpr (BOTH) {
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                if (row0 + i >= p.rows) continue;
                const float r = 1.0f / rs[i];
                uint32_t out[VEC / 4];
#pragma unroll
                for (int k = 0; k < VEC / 4; ++k) {
                    const uint32_t e[4] = {elem(i, 4 * k), elem(i, 4 * k + 1), elem(i, 4 * k + 2),
                                           elem(i, 4 * k + 3)};
                    out[k] = cast4<FMT>(e, rs[i], r, nf);
                }
                uint8_t *dst = p.codes + (row0 + i) * p.cols + col0;
                if constexpr (VEC == 8) *reinterpret_cast<u32x2 *>(dst) = u32x2{out[0], out[1]};
                else *reinterpret_cast<uint32_t *>(dst) = out[0];
            }
        }
        __syncthreads();
        // 8 lanes per transposed row, 16 bytes each
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = q * 32 + (tid >> 3), piece = tid & 7;
            const int key = (c / VEC) & (UNITS - 1);
            u32x4 v;
            if constexpr (WPU == 2) {
                const u32x2 lo = *reinterpret_cast<const u32x2 *>(&codes_lds[c * 32 + ((2 * piece) ^ key) * 2]);
                const u32x2 hi = *reinterpret_cast<const u32x2 *>(&codes_lds[c * 32 + ((2 * piece + 1) ^ key) * 2]);
                v = u32x4{lo.x, lo.y, hi.x, hi.y};
            } else {
                v = *reinterpret_cast<const u32x4 *>(&codes_lds[c * 32 + (piece ^ key) * 4]);
            }
            const int64_t col = tc * 128 + c;
            if (col < p.cols)
                *reinterpret_cast<u32x4 *>(p.codes_t + col * p.rows_pad + tr * 128 + piece * 16) = v;
        }
        __syncthreads();                              // LDS is reused by the next tile
    }
    if (saw_nf && p.nonfinite) *p.nonfinite = 1;
}

template <int FMT, bool TILE, bool BOTH>
hipError_t launch(const void *x, gs_dtype dt, const TransposeArgs &p, hipStream_t stream) {
    const dim3 grid((uint32_t)(p.ntiles < GS_MAX_GRID ? p.ntiles : GS_MAX_GRID));
    if (dt == GS_BF16)
        hipLaunchKernelGGL((quant_transposed_kernel<FMT, TILE, BOTH, uint16_t>), grid, dim3(256), 0,
                           stream, static_cast<const uint16_t *>(x), p);
    else
        hipLaunchKernelGGL((quant_transposed_kernel<FMT, TILE, BOTH, float>), grid, dim3(256), 0,
                           stream, static_cast<const float *>(x), p);
    return hipGetLastError();
}

inline bool misaligned(const void *p, uintptr_t a) { return (uintptr_t(p) & (a - 1)) != 0; }

}  // namespace

}  // namespace gsk

extern "C" gs_status fp8_quantize_transposed(const void *x, gs_dtype x_dtype, int64_t rows,
                                             int64_t cols, fp8_format fmt, fp8_granularity g,
                                             uint8_t *codes_t, float *scales_t, uint8_t *codes,
                                             float *scales, int32_t *nonfinite, void *stream) {
    using namespace gsk;
    constexpr int64_t kMaxDim = int64_t(1) << 31, kMaxElems = int64_t(1) << 40;
    if (x_dtype != GS_BF16 && x_dtype != GS_F32) return GS_ERR_DTYPE;
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2) return GS_ERR_ARG;
    if (g != FP8_BLOCK_1x128 && g != FP8_BLOCK_128x128) return GS_ERR_ARG;
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim || rows * cols > kMaxElems)
        return GS_ERR_SIZE;
    const bool tile = g == FP8_BLOCK_128x128, both = codes || scales;
    if (tile && (rows % 128 != 0 || cols % 128 != 0)) return GS_ERR_SHAPE;
    if (both && cols % 128 != 0) return GS_ERR_SHAPE;
    if (rows * cols > 0 && (!x || !codes_t || !scales_t)) return GS_ERR_NULL;
    if (both && (!codes || !scales)) return GS_ERR_NULL;
    if (misaligned(x, 16) || misaligned(codes_t, 16) || misaligned(codes, 16) ||
        misaligned(scales_t, 4) || misaligned(scales, 4) || misaligned(nonfinite, 4))
        return GS_ERR_ALIGN;
    if (rows == 0 || cols == 0) return GS_OK;
    TransposeArgs p{};
    p.rows = rows;
    p.cols = cols;
    p.tiles_r = (rows + 127) / 128;
    p.rows_pad = p.tiles_r * 128;
    p.ntiles = p.tiles_r * ((cols + 127) / 128);
    p.codes_t = codes_t;
    p.scales_t = scales_t;
    p.codes = codes;
    p.scales = scales;
    p.nonfinite = nonfinite;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    switch ((fmt == FP8_E5M2) | tile << 1 | both << 2) {
        case 0: e = launch<0, false, false>(x, x_dtype, p, s); break;
        case 1: e = launch<1, false, false>(x, x_dtype, p, s); break;
        case 2: e = launch<0, true, false>(x, x_dtype, p, s); break;
        case 3: e = launch<1, true, false>(x, x_dtype, p, s); break;
        case 4: e = launch<0, false, true>(x, x_dtype, p, s); break;
        case 5: e = launch<1, false, true>(x, x_dtype, p, s); break;
        case 6: e = launch<0, true, true>(x, x_dtype, p, s); break;
        default: e = launch<1, true, true>(x, x_dtype, p, s); break;
    }
    return e == hipSuccess ? GS_OK : GS_ERR_HIP;
}

// quant.hip -- 8-bit codes (e4m3) of a matrix's rows with a binary32 scale for
// each block of 128 elements.
//
//   s = max|x| / 448,  r = min(448 (1 / max|x|), largest binary32),  code = RNE(clamp(x r))
//
// A block belongs to 8 neighbouring lanes, 16 elements each: two 16-byte loads
// (16-bit types), a maximum over 8 lanes, one 16-byte store.  Bound by bytes:
// one read, one write of half of it.  On MI355X 8192 x 8192 in bf16 (203 MB) take 36.4 to
// 37.3 us, 5.5 TB/s: above the rate of a large copy (4.85), as a third of the traffic is
// writes and not half; in binary32 (338 MB) 59.6 us, 5.7 TB/s; 32 x 4096 take 3 us, which is
// the launch.
#include <algorithm>

#include "layer_device.h"

namespace mpp {
namespace layer {
namespace {

constexpr int kBlock = 256;
constexpr float kTop = 448.0f;

template <int T>
__global__ void __launch_bounds__(kBlock) k_quant(QuantArgs a, size_t items) {
    const size_t flat = static_cast<size_t>(blockIdx.x) * kBlock + threadIdx.x;
    const size_t item = flat >> 3;                // (row, block)
    const unsigned j = flat & 7;
    if (item >= items) return;
    const size_t row = item / a.blocks;
    const unsigned block = static_cast<unsigned>(item - row * a.blocks);
    const unsigned col = block * AR_F8_BLOCK + j * 16;
    const bool active = col < a.cols;
    float x[16];
    unsigned top = 0;
    if (active) {
        load_n<T, 8>(a.x, row * a.x_row + col, x);
        load_n<T, 8>(a.x, row * a.x_row + col + 8, x + 8);
        // magnitudes compare as integers, a NaN above everything
#pragma unroll
        for (int e = 0; e < 16; ++e) top = max(top, __builtin_bit_cast(unsigned, x[e]) & 0x7FFFFFFFu);
    }
    for (int step = 1; step < 8; step <<= 1) top = max(top, static_cast<unsigned>(__shfl_xor(static_cast<int>(top), step)));
    const float peak = __builtin_bit_cast(float, top);
    // one IEEE division each; a NaN peak leaves factor 0, so only the NaN's own code is one
    const float factor = peak > 0.0f ? fminf(kTop * (1.0f / peak), 3.4028234663852886e38f) : 0.0f;
    if (!active) return;
    unsigned w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float p = x[4 * e + i] * factor;
            // a comparison keeps a NaN, which the conversion turns to the NaN code
            y[i] = p > kTop ? kTop : p < -kTop ? -kTop : p;
        }
        int u = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        u = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], u, true);
        w[e] = static_cast<unsigned>(u);
    }
    *reinterpret_cast<v4u *>(a.codes + row * a.codes_row + col) = v4u{w[0], w[1], w[2], w[3]};
    if (j == 0) a.scales[row * a.blocks + block] = peak / kTop;
}

template <int T>
hipError_t launch_t(const QuantArgs &all, hipStream_t stream) {
    // a launch holds fewer than 2^32 lanes: longer calls go by ranges of rows
    const size_t most = std::max<size_t>(1, (size_t(1) << 28) / all.blocks);
    for (size_t r0 = 0; r0 < all.rows; r0 += most) {
        QuantArgs a = all;
        a.rows = std::min(most, all.rows - r0);
        a.x = static_cast<const char *>(all.x) + r0 * all.x_row * (T == AR_F32 ? 4 : 2);
        a.codes = all.codes + r0 * all.codes_row;
        a.scales = all.scales + r0 * all.blocks;
        const size_t items = a.rows * a.blocks;
        const size_t grid = (items * 8 + kBlock - 1) / kBlock;
        hipLaunchKernelGGL((k_quant<T>), dim3(static_cast<unsigned>(grid)), dim3(kBlock), 0, stream, a, items);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_quant(const QuantArgs &a, ar_dtype type, hipStream_t stream) {
    if (type == AR_F32) return launch_t<AR_F32>(a, stream);
    if (type == AR_F16) return launch_t<AR_F16>(a, stream);
    return launch_t<AR_BF16>(a, stream);
}

}  // namespace layer
}  // namespace mpp

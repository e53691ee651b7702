// qk.hip -- norm of each head's queries and keys and the position rotation in
// one pass over the data.
//
//   y = x * (1 / sqrt(mean(x^2) + eps)) * w
//   (a, b) -> (a cos - b sin, b cos + a sin)
//
// A head's head_dim elements belong to G neighbouring lanes of a wave (G a
// power of two), 2 * CH elements a lane: the lane that holds elements i .. i +
// CH - 1 also holds their partners (rot_dim / 2 further, or the next ones where
// pairs are interleaved), so the turn needs no exchange between lanes and the
// mean of squares is a sum over G lanes.  Everything between the load and the
// one rounding at the store is binary32.
//
// Bound by bytes: every element is read once and written once.  The angles'
// rows are shared by all heads of a token and come from the caches.  On MI355X 2048
// tokens of 32 and 8 heads of 128 in bf16 (51 MB with the angles) take 11.6 us, 4.4
// TB/s where a large copy reaches 4.85, and 21.7 in binary32 (103 MB, 4.7 TB/s); 32 tokens
// take 4 us, which is the launch.
#include <algorithm>

#include "layer_device.h"

namespace mpp {
namespace layer {
namespace {

constexpr int kBlock = 256;

template <int T, int CH, bool INTERLEAVED>
__global__ void __launch_bounds__(kBlock) k_qk(QkArgs a, unsigned lanes_log, unsigned items) {
    const unsigned lanes = 1u << lanes_log;
    const unsigned flat = blockIdx.x * kBlock + threadIdx.x;
    const unsigned item = flat >> lanes_log;      // (token, head)
    const unsigned j = flat & (lanes - 1);        // lane within the head
    if (item >= items) return;                    // whole groups of lanes leave together
    const unsigned token = item / a.heads_all;
    const unsigned head = item - token * a.heads_all;

    // chunks of CH elements; the turning ones come in pairs
    const unsigned turning = a.rot_dim / (2 * CH);
    const bool active = j < a.head_dim / (2 * CH);
    unsigned at0, at1;
    if (!INTERLEAVED && j < turning) {
        at0 = j * CH;
        at1 = at0 + a.rot_dim / 2;
    } else {
        at0 = 2 * j * CH;
        at1 = at0 + CH;
    }

    const bool is_q = head < a.heads_q;
    const bool is_v = head >= a.heads_q + a.heads_kv;
    size_t row = token;
    if (!is_q && a.slots != nullptr) {
        const long long slot = a.slots[token];
        if (slot < 0 || static_cast<size_t>(slot) >= a.cache_rows) return;
        row = static_cast<size_t>(slot);
    }
    const void *src;
    void *dst;
    const void *weight;
    size_t from, to;
    if (is_q) {
        src = a.q;
        dst = a.q_out;
        weight = a.q_weight;
        from = token * a.q_token + head * a.q_head;
        to = row * a.q_out_token + head * a.q_out_head;
    } else if (!is_v) {
        const unsigned h = head - a.heads_q;
        src = a.k;
        dst = a.k_out;
        weight = a.k_weight;
        from = token * a.k_token + h * a.k_head;
        to = row * a.k_out_token + h * a.k_out_head;
    } else {
        const unsigned h = head - a.heads_q - a.heads_kv;
        src = a.v;
        dst = a.v_out;
        weight = nullptr;
        from = token * a.v_token + h * a.v_head;
        to = row * a.v_out_token + h * a.v_out_head;
    }

    float x[2 * CH];
    if (active) {
        load_n<T, CH>(src, from + at0, x);
        load_n<T, CH>(src, from + at1, x + CH);
    } else {
#pragma unroll
        for (int e = 0; e < 2 * CH; ++e) x[e] = 0.0f;
    }
    if (!is_v) {
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 2 * CH; ++e) sum = __builtin_fmaf(x[e], x[e], sum);
        for (unsigned step = 1; step < lanes; step <<= 1) sum += __shfl_xor(sum, step);
        const float inv = 1.0f / sqrtf(__builtin_fmaf(sum, a.inv_dim, a.eps));
        if (active && weight != nullptr) {
            float w[2 * CH];
            load_n<T, CH>(weight, at0, w);
            load_n<T, CH>(weight, at1, w + CH);
#pragma unroll
            for (int e = 0; e < 2 * CH; ++e) x[e] = x[e] * inv * w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 2 * CH; ++e) x[e] *= inv;
        }
        if (turning != 0) {
            const long long p = a.positions[token];
            if (p < 0 || static_cast<size_t>(p) >= a.table_rows) {
#pragma unroll
                for (int e = 0; e < 2 * CH; ++e) x[e] = __builtin_nanf("");
            } else if (j < turning) {
                const float *t = a.table + static_cast<size_t>(p) * a.rot_dim;
                float c[CH], s[CH];
                load_n<AR_F32, CH>(t, j * CH, c);
                load_n<AR_F32, CH>(t, a.rot_dim / 2 + j * CH, s);
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    const int ia = INTERLEAVED ? 2 * e : e;
                    const int ib = INTERLEAVED ? 2 * e + 1 : CH + e;
                    const float xa = x[ia], xb = x[ib];
                    x[ia] = __builtin_fmaf(xa, c[e], -(xb * s[e]));
                    x[ib] = __builtin_fmaf(xb, c[e], xa * s[e]);
                }
            }
        }
    }
    if (active) {
        store_n<T, CH>(dst, to + at0, x);
        store_n<T, CH>(dst, to + at1, x + CH);
    }
}

template <int T, int CH>
hipError_t launch_ch(const QkArgs &all, bool interleaved, hipStream_t stream) {
    const unsigned per_head = all.head_dim / (2 * CH);
    unsigned lanes_log = 0;
    while ((1u << lanes_log) < per_head) ++lanes_log;
    const unsigned per_block = kBlock >> lanes_log;
    // a launch holds fewer than 2^32 lanes: longer calls go by ranges of tokens
    const unsigned most = std::max(1u, (1u << (31 - lanes_log)) / all.heads_all);
    constexpr size_t kSize = T == AR_F32 ? 4 : 2;
    for (unsigned t0 = 0; t0 < all.tokens; t0 += most) {
        QkArgs a = all;
        a.tokens = std::min(most, all.tokens - t0);
        const auto from = [&](const void *p, size_t stride) {
            return p == nullptr ? nullptr : static_cast<const char *>(p) + t0 * stride * kSize;
        };
        a.q = from(all.q, all.q_token);
        a.k = from(all.k, all.k_token);
        a.v = from(all.v, all.v_token);
        a.q_out = const_cast<char *>(from(all.q_out, all.q_out_token));
        if (all.slots == nullptr) {
            a.k_out = const_cast<char *>(from(all.k_out, all.k_out_token));
            a.v_out = const_cast<char *>(from(all.v_out, all.v_out_token));
        } else {
            a.slots = all.slots + t0;
        }
        if (all.positions != nullptr) a.positions = all.positions + t0;
        const unsigned items = a.tokens * a.heads_all;
        const unsigned grid = (items + per_block - 1) / per_block;
        if (interleaved) {
            hipLaunchKernelGGL((k_qk<T, CH, true>), dim3(grid), dim3(kBlock), 0, stream, a, lanes_log, items);
        } else {
            hipLaunchKernelGGL((k_qk<T, CH, false>), dim3(grid), dim3(kBlock), 0, stream, a, lanes_log, items);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int T>
hipError_t launch_t(const QkArgs &a, bool interleaved, hipStream_t stream) {
    // 16-byte accesses of 16-bit elements where the sizes allow them
    if (a.head_dim % 16 == 0 && a.rot_dim % 16 == 0) return launch_ch<T, 8>(a, interleaved, stream);
    return launch_ch<T, 4>(a, interleaved, stream);
}

}  // namespace

hipError_t launch_qk(const QkArgs &a, ar_dtype type, bool interleaved, hipStream_t stream) {
    if (type == AR_F32) return launch_t<AR_F32>(a, interleaved, stream);
    if (type == AR_F16) return launch_t<AR_F16>(a, interleaved, stream);
    return launch_t<AR_BF16>(a, interleaved, stream);
}

}  // namespace layer
}  // namespace mpp

// attn.hip -- attention of packed sequences over a prompt or a cache, causal or
// whole, with grouped heads.
//
//   out_i = sum_j softmax_j(scale q_i.k_j) v_j          over the seen j
//
// One pass over the keys with a running reference m and sum l per query:
// p = 2^(c s - c m), c = scale log2(e).  The queries of all heads that share a
// key head are packed into one row index, r = token * group + head, so a tile of
// rows reads each key once for the whole group.
//
// Scores are computed transposed, S^T = K Q^T with the 32x32x16 instruction: a
// lane then holds one query (column l % 32) and 16 of 32 keys, so the softmax
// statistics are one register per lane and a maximum over a row costs one
// exchange between lane halves.  P^T in that layout is already the second operand
// of O^T += V^T P^T: its depth slots p = 0..7 of lane half h hold keys 4h + p
// (p < 4) and 4h + 8 + p - 4, and V^T is read from LDS with the transposing
// reads in the same order.
//
// The probabilities are rounded to the type there, half a step each, since the instruction
// multiplies nothing wider at this rate; the sum that divides them keeps binary32.  Against
// 64 bits, 2048 and 8192 tokens in bfloat16 are off by 2.0e-3 of the result's norm, where
// the rounding of the result alone leaves 1.6e-3.
//
// LDS tiles hold rows of DB elements in 16-byte chunks whose slots are permuted
// per row, keys by chunk ^ row (16-byte reads of eight rows at one chunk), values
// by pairs of chunks (transposing reads of four rows at 32 bytes), so that reads
// spread over all banks.  Chunks past head_dim and rows past the sequence are
// zeros (out of the buffer's range).
#include <algorithm>

#include "layer_device.h"

namespace mpp {
namespace layer {
namespace {

constexpr unsigned kOut = 0x80000000u;   // an offset past every buffer: reads zeros
constexpr float kNone = -__builtin_inff();
constexpr float kLn2 = 0.69314718055994530942f;
// The sums are rescaled when a row's maximum outgrows its reference by more than this
// many powers of two: until then the probabilities stay below 2^8, in range for every
// type and no less exact.
constexpr float kSlack = 8.0f;
// Probabilities meet the values in the type, whose range is binary16's least: taken 2^7 times
// as large, at most 2^15 with the slack, they keep what lies down to 2^-32 of the reference (without,
// to 2^-25: 30000 keys at 2^-26 of one other's probability were lost altogether).  The sums of
// a row have the factor too; it is a part of the reference that goes with them.
template <int T>
constexpr float kLift = T == AR_F16 ? 7.0f : 0.0f;

template <int T>
struct Mat;
template <>
struct Mat<AR_BF16> {
    typedef v8bf frag;
    static LAYER_DEV v16f mul(v8bf x, v8bf y, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0); }
};
template <>
struct Mat<AR_F16> {
    typedef v8h frag;
    static LAYER_DEV v16f mul(v8h x, v8h y, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, c, 0, 0, 0); }
};

// A value of both lane halves: the lower half's and the upper's.  (Elements are
// copied to scalars before the cast: a bit cast of a vector's element reads element 0.)
struct Halves {
    float low, high;
};
LAYER_DEV Halves halves(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned low = r[0], high = r[1];
    return Halves{__builtin_bit_cast(float, low), __builtin_bit_cast(float, high)};
}
LAYER_DEV float max_halves(float x) {
    const Halves h = halves(x);
    return fmaxf(h.low, h.high);
}
LAYER_DEV float sum_halves(float x) {
    const Halves h = halves(x);
    return h.low + h.high;
}

// One sequence as a workgroup sees it; bounds cut to the tensors.
struct Seq {
    long long q0, k0;
    int len_q, len_k;
};
LAYER_DEV int queries(const AttnArgs &a, int b, long long &q0) {
    long long q1 = a.cu_q[b + 1];
    q0 = a.cu_q[b];
    q0 = q0 < 0 ? 0 : q0 > a.total_q ? a.total_q : q0;
    q1 = q1 < q0 ? q0 : q1 > a.total_q ? a.total_q : q1;
    return static_cast<int>(q1 - q0 < a.max_q ? q1 - q0 : a.max_q);
}
LAYER_DEV Seq sequence(const AttnArgs &a, int b) {
    Seq s;
    s.len_q = queries(a, b, s.q0);
    const long long k0 = a.k_start[b];
    long long n = a.k_len[b];
    if (k0 < 0 || k0 > a.rows_k || n < 0) n = 0;
    if (n > 0 && n > a.rows_k - k0) n = a.rows_k - k0;
    if (n > a.max_k) n = a.max_k;
    s.k0 = n > 0 ? k0 : 0;
    s.len_k = static_cast<int>(n);
    return s;
}

// A wave's view of its 32 rows and their running sums.
template <int T, int DB>
struct Rows {
    typename Mat<T>::frag q[DB / 16];
    v16f o[DB / 32];
    float m, l;        // reference (raw score) and this lane's share of the sum
    int limit;         // last key this lane's row sees
};

// Queries of rows row0 .. row0 + 31 of key head `head`.
template <int T, int DB>
LAYER_DEV void start_rows(const AttnArgs &a, const Seq &s, int head, int row0, Rows<T, DB> &w) {
    const unsigned lane = threadIdx.x & 63;
    const int last = s.len_q * a.group - 1;
    const int r = min(row0 + static_cast<int>(lane & 31), last);
    const int token = r / a.group, sub = r - token * a.group;
    const uint16_t *p = static_cast<const uint16_t *>(a.q) + static_cast<size_t>(s.q0 + token) * a.q_token +
                        static_cast<size_t>(head * a.group + sub) * a.q_head;
#pragma unroll
    for (int i = 0; i < DB / 16; ++i) {
        const int d = i * 16 + static_cast<int>(lane >> 5) * 8;
        v4u u = {0, 0, 0, 0};
        if (d < a.head_dim) u = *reinterpret_cast<const v4u *>(p + d);
        w.q[i] = __builtin_bit_cast(typename Mat<T>::frag, u);
    }
#pragma unroll
    for (int i = 0; i < DB / 32; ++i) {
#pragma unroll
        for (int e = 0; e < 16; ++e) w.o[i][e] = 0.0f;
    }
    w.m = kNone;
    w.l = 0.0f;
    w.limit = s.len_k - 1;
    if (a.causal) w.limit = min(w.limit, token + s.len_k - s.len_q);
}

// Last key that any of rows 0 .. row (one row each, not a lane's) sees.
LAYER_DEV int limit_of(const AttnArgs &a, const Seq &s, int row) {
    row = min(row, s.len_q * a.group - 1);
    return a.causal ? min(s.len_k - 1, row / a.group + s.len_k - s.len_q) : s.len_k - 1;
}

// How the chunks of a row of values are permuted: four rows at 64 bytes each (what half
// a wave reads transposed) cover all banks.
template <int DB>
LAYER_DEV unsigned pair_twist(unsigned row) {
    return DB == 64 ? (row & 2) << 1 : (row & 3) << 2;
}

// Loads of KT rows of keys (PAIRS false) or values (true) to LDS by W waves, of
// which this is number `wave`: rows j0 .. of a sequence of len rows.  ROLLED: one
// instruction in a loop (the compiler follows only the first few loads to LDS in a kernel
// one by one; later ones it waits for all together).
template <int DB, int KT, int W, bool PAIRS, bool ROLLED = false>
LAYER_DEV void fill(char *tile, const uint16_t *base, size_t stride, int j0, int len, int dim, int wave) {
    constexpr int kChunks = DB / 8;             // 16-byte chunks of a row
    constexpr int kRows = 64 / kChunks;         // rows a wave loads at once
    constexpr int kEach = KT / kRows / W;
    constexpr unsigned kMask = kChunks < 16 ? kChunks - 1 : 15;
    const unsigned lane = threadIdx.x & 63;
    const int have = min(KT, len - j0);
    const unsigned bytes = static_cast<unsigned>(stride * 2);
    const auto buf = buffer_of(base + static_cast<size_t>(j0) * stride,
                               static_cast<int>(static_cast<unsigned>(have - 1) * bytes + static_cast<unsigned>(dim) * 2));
    const unsigned in = lane / kChunks, slot = lane % kChunks;
    const auto part = [&](int i) __attribute__((always_inline)) {
        const unsigned p = static_cast<unsigned>(wave * kEach + i), row = p * kRows + in;
        const unsigned chunk = PAIRS ? slot ^ pair_twist<DB>(row) : slot ^ (row & kMask);
        const unsigned past = chunk * 8 < static_cast<unsigned>(dim) ? 0u : kOut;
        load_lds16(buf, tile + p * 1024, (in * bytes + chunk * 16) | past, p * kRows * bytes);
    };
    if constexpr (ROLLED) {
#pragma nounroll
        for (int i = 0; i < kEach; ++i) part(i);
    } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i) part(i);
    }
}

// A value that only later queries see must not reach the earlier ones of its tile,
// but in the product 0 times an infinity or a NaN would.  So in the tiles that some
// row does not wholly see such values are replaced by zeros in LDS, and after the
// last tile the rows that do see them add them to their sums.
template <int T>
struct Bits;
template <>
struct Bits<AR_BF16> {
    static constexpr unsigned kExp = 0x7F80u, kLow = 0x80u;
};
template <>
struct Bits<AR_F16> {
    static constexpr unsigned kExp = 0x7C00u, kLow = 0x400u;
};

// Bit 15 of each half that is not finite (the sum carries there where the exponent is all ones).
template <int T>
LAYER_DEV unsigned not_finite(unsigned u) {
    return ((u & (Bits<T>::kExp * 0x10001u)) + Bits<T>::kLow * 0x10001u) & 0x80008000u;
}

// Replaces them in an LDS tile of `bytes` bytes, shared by `lanes` lanes of which
// this is number `lane`; whether this lane found one.
template <int T>
LAYER_DEV bool clear_not_finite(char *tile, int bytes, int lane, int lanes) {
    unsigned found = 0;
    for (int at = lane * 16; at < bytes; at += lanes * 16) {
        v4u *p = reinterpret_cast<v4u *>(tile + at);
        v4u u = *p;
        unsigned here = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned bad = not_finite<T>(u[e]);
            here |= bad;
            u[e] &= ~(((bad >> 15) & 0x10001u) * 0xFFFFu);
        }
        if (here != 0) *p = u;
        found |= here;
    }
    return found != 0;
}

// Adds what keys j0 .. j1 - 1 had of them to the rows that see them.
template <int T, int DB>
LAYER_DEV void add_not_finite(const uint16_t *v, size_t stride, int j0, int j1, int dim, Rows<T, DB> &w) {
    const int half = static_cast<int>(threadIdx.x >> 5) & 1;
#pragma nounroll
    for (int j = j0; j < j1; ++j) {
        if (j > w.limit) continue;
#pragma unroll
        for (int i = 0; i < DB / 8; ++i) {
            const int d = i * 8 + half * 4;
            if (d >= dim) continue;
            const v2u u = *reinterpret_cast<const v2u *>(v + static_cast<size_t>(j) * stride + d);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const v2f f = unpack2<T>(u[e]);
                const unsigned bad = not_finite<T>(u[e]);
                if ((bad & 0x8000u) != 0) w.o[i / 4][(i % 4) * 4 + 2 * e] += f.x;
                if ((bad >> 31) != 0) w.o[i / 4][(i % 4) * 4 + 2 * e + 1] += f.y;
            }
        }
    }
}

// Raw scores of one tile of KT keys against the wave's rows.
template <int T, int DB, int KT>
LAYER_DEV void tile_scores(const char *ks, const Rows<T, DB> &w, v16f (&s)[KT / 32]) {
    typedef typename Mat<T>::frag Frag;
    constexpr int kRow = DB * 2;
    constexpr unsigned kMask = DB / 8 < 16 ? DB / 8 - 1 : 15;
    const unsigned lane = threadIdx.x & 63, half = lane >> 5;
#pragma unroll
    for (int t = 0; t < KT / 32; ++t) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < DB / 16; ++i) {
#pragma unroll
        for (int t = 0; t < KT / 32; ++t) {
            const unsigned row = t * 32 + (lane & 31), chunk = (2 * i + half) ^ (row & kMask);
            const Frag k = __builtin_bit_cast(Frag, *reinterpret_cast<const v4u *>(ks + row * kRow + chunk * 16));
            s[t] = Mat<T>::mul(k, w.q[i], s[t]);
        }
    }
}

// The largest score of each row (both lane halves have it).
template <int KT>
LAYER_DEV float tile_top(const v16f (&s)[KT / 32]) {
    float top = s[0][0];
#pragma unroll
    for (int t = 0; t < KT / 32; ++t) {
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[t][e]);
    }
    return max_halves(top);
}

// Probabilities p up to the rows' references, and their sums.
template <int T, int DB, int KT>
LAYER_DEV void tile_powers(const v16f (&s)[KT / 32], float c, Rows<T, DB> &w, typename Mat<T>::frag (&p)[KT / 16]) {
    const float mc = (w.m == kNone ? 0.0f : w.m * c) - kLift<T>;
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < KT / 32; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v4u u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][8 * h + 2 * e], c, -mc));
                const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][8 * h + 2 * e + 1], c, -mc));
                sum += x + y;
                u[e] = pack2<T>(x, y);
            }
            p[2 * t + h] = __builtin_bit_cast(typename Mat<T>::frag, u);
        }
    }
    w.l += sum;
}

// Any tile: keys past a row's limit left out, the references moved to the rows' new
// maxima and the sums with them.
template <int T, int DB, int KT>
LAYER_DEV void tile_general(const char *ks, int j0, int free_to, float c, Rows<T, DB> &w, typename Mat<T>::frag (&p)[KT / 16]) {
    const unsigned lane = threadIdx.x & 63, half = lane >> 5;
    v16f s[KT / 32];
    tile_scores<T, DB, KT>(ks, w, s);
    if (j0 + KT - 1 > free_to) {   // some row of the wave does not see all of it
        const int base = j0 + static_cast<int>(half) * 4;
#pragma unroll
        for (int t = 0; t < KT / 32; ++t) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int j = base + t * 32 + 8 * (e / 4) + e % 4;
                s[t][e] = j <= w.limit ? s[t][e] : kNone;
            }
        }
    }
    const float m = fmaxf(w.m, tile_top<KT>(s));
    const float mc = m == kNone ? 0.0f : m * c;
    const float shrink = __builtin_amdgcn_exp2f(__builtin_fmaf(w.m, c, -mc));
    w.m = m;
    w.l *= shrink;
#pragma unroll
    for (int i = 0; i < DB / 32; ++i) {
#pragma unroll
        for (int e = 0; e < 16; ++e) w.o[i][e] *= shrink;
    }
    tile_powers<T, DB, KT>(s, c, w, p);
}

// Fragment (i, h) of V^T: 32 elements of the rows by 16 keys.
template <int T, int DB>
LAYER_DEV typename Mat<T>::frag value_fragment(const char *vs, int i, int h) {
    constexpr int kRow = DB * 2;
    const unsigned lane = threadIdx.x & 63, half = lane >> 5;
    const unsigned i16 = lane & 15;
    const unsigned row = half * 4 + (i16 >> 2);
    const unsigned twist = pair_twist<DB>(row);     // (the steps add multiples of 8 rows)
    const unsigned chunk = i * 4 + ((lane >> 4) & 1) * 2 + ((i16 & 3) >> 1);
    const char *at = vs + row * kRow + ((chunk ^ twist) << 4) + (i16 & 1) * 8;
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(at + h * 16 * kRow));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(at + (h * 16 + 8) * kRow));
    return __builtin_bit_cast(typename Mat<T>::frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// O^T += V^T P^T for one tile.
template <int T, int DB, int KT>
LAYER_DEV void tile_values(const char *vs, Rows<T, DB> &w, const typename Mat<T>::frag (&p)[KT / 16]) {
#pragma unroll
    for (int i = 0; i < DB / 32; ++i) {
#pragma unroll
        for (int h = 0; h < KT / 16; ++h) w.o[i] = Mat<T>::mul(value_fragment<T, DB>(vs, i, h), p[h], w.o[i]);
    }
}

// The same for the tile before and, under its products, the probabilities of this one,
// which take the other's place.  The scheduling barriers keep a few of the one between
// two of the other; left alone the compiler puts all products first.
template <int T, int DB, int KT>
LAYER_DEV void tile_both(const char *vs, v16f (&s)[KT / 32], float c, Rows<T, DB> &w, typename Mat<T>::frag (&p)[KT / 16]) {
    constexpr int kFrags = DB / 32, kScores = 8 / kFrags;   // of a step of 16 keys, beside each product
    typename Mat<T>::frag v[2][kFrags];
#pragma unroll
    for (int i = 0; i < kFrags; ++i) v[0][i] = value_fragment<T, DB>(vs, i, 0);
    const float mc = (w.m == kNone ? 0.0f : w.m * c) - kLift<T>;
    float sum = 0.0f;
#pragma unroll
    for (int h = 0; h < KT / 16; ++h) {
        if (h + 1 < KT / 16) {
#pragma unroll
            for (int i = 0; i < kFrags; ++i) v[(h + 1) & 1][i] = value_fragment<T, DB>(vs, i, h + 1);
        }
        float x[8];
#pragma unroll
        for (int i = 0; i < kFrags; ++i) {
            w.o[i] = Mat<T>::mul(v[h & 1][i], p[h], w.o[i]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = i * kScores; e < (i + 1) * kScores; ++e) {
                x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[h / 2][8 * (h & 1) + e], c, -mc));
                sum += x[e];
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        v4u u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = pack2<T>(x[2 * e], x[2 * e + 1]);
        p[h] = __builtin_bit_cast(typename Mat<T>::frag, u);
    }
    w.l += sum;
}

// Log of a row's sum, from the reference in powers of two and the sum.
LAYER_DEV float log_sum(float mc, float l) { return l == 0.0f ? kNone : (mc + log2f(l)) * kLn2; }

// What one lane has, for the whole wave.
LAYER_DEV long long lane_of(long long v, int lane) {
    const int low = __builtin_amdgcn_readlane(static_cast<int>(v), lane);
    const int high = __builtin_amdgcn_readlane(static_cast<int>(v >> 32), lane);
    return static_cast<long long>(high) << 32 | static_cast<unsigned>(low);
}
LAYER_DEV Seq lane_of(const Seq &s, int lane) {
    return Seq{lane_of(s.q0, lane), lane_of(s.k0, lane), __builtin_amdgcn_readlane(s.len_q, lane),
               __builtin_amdgcn_readlane(s.len_k, lane)};
}

// Sums of v over the lanes up to each, all of the wave's being active.
template <int CTRL, int ROWS>
LAYER_DEV int moved(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
LAYER_DEV int sums_to(int v) {
    v += moved<0x111, 0xF>(v);   // from one lane below in the row of 16, then two, four, eight
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);   // the last lane of the row below
    v += moved<0x143, 0xC>(v);   // lane 31
    return v;
}

// Tile i of a call whose sequences differ in length: of all sequences' tiles of 128 rows
// the ones that see most keys, in steps of 64, first.  False past the last.  A lane counts
// the tiles of every 64th sequence, the number of steps is found by halving.
LAYER_DEV bool gathered_tile(const AttnArgs &a, int i, Seq &seq, int &tile) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    const auto of = [&](int b) { return b < a.batch ? sequence(a, b) : Seq{0, 0, 0, 0}; };
    // how many of a sequence's tiles take u steps or more: its last ones
    const auto having = [&](const Seq &x, int u) {
        const int tiles = (x.len_q * a.group + 127) / 128;
        if (u == 0) return tiles;
        const int key = (u - 1) * 64;   // the first of the step
        if (key >= x.len_k) return 0;
        const int token = a.causal ? key - (x.len_k - x.len_q) : 0;   // the first that sees it
        if (token <= 0) return tiles;
        return token < x.len_q ? tiles - token * a.group / 128 : 0;
    };
    const Seq first = of(lane);
    const auto from = [&](int u) {
        int n = having(first, u);
        for (int b = 64; b < a.batch; b += 64) n += having(of(b + lane), u);
        return __builtin_amdgcn_readlane(sums_to(n), 63);
    };
    if (i >= from(0)) return false;
    int low = 0, high = (a.max_k + 63) / 64 + 1;   // from(low) > i >= from(high)
    while (high - low > 1) {
        const int mid = (low + high) / 2;
        if (from(mid) > i) {
            low = mid;
        } else {
            high = mid;
        }
    }
    int rank = i - from(low + 1);
    for (int b = 0; b < a.batch; b += 64) {
        const Seq x = b == 0 ? first : of(b + lane);
        const int many = having(x, low), n = many - having(x, low + 1), to = sums_to(n);
        const unsigned long long past = __ballot(to > rank);
        if (past != 0) {
            const int in = __ffsll(past) - 1;
            seq = lane_of(x, in);
            tile = __builtin_amdgcn_readlane(having(x, 0) - many + rank - (to - n), in);
            return true;
        }
        rank -= __builtin_amdgcn_readlane(to, 63);
    }
    return false;
}

// Prompts: tiles of 128 rows, four waves of 32 rows each for every one of S streams;
// stream g takes tiles g, g + S, ... of 64 keys.  With two streams a tile of rows
// is done in half the time, which counts where a call has few of them.  Everyone of a
// workgroup meets once for every S tiles of keys.
// Bound by the matrix cores and the exponentials beside them: 8192 tokens, 32 heads over 8
// of 128, causal, take 506 to 515 us, 1.07 PFLOP/s (the first calls after a rest 530 and
// more), where a large bf16 product reaches 1.2; the matrix cores are busy for 60 % of the
// cycles, and a score costs as many cycles of the vector unit as of theirs.  Short calls are bound by the chain of a row's tiles (1.4 us each
// alone, about 1 with a second workgroup on the CU) and 5 us for beginning and end: 2048
// tokens take 47 to 48 us.
template <int T, int DB, int S>
__global__ void __launch_bounds__(256 * S, DB <= 128 ? 2 / S : 1) k_attn_rows(AttnArgs a, unsigned tiles, bool gathered) {
    constexpr int KT = 64;
    constexpr int kTile = KT * DB * 2;
    // Whether a step multiplies the values of the tile before, under which it finds its own
    // probabilities, or its own tile's.  (us so and not, 32 heads over 8, 2048 tokens of 128: 49.4
    // and 52.9; 8 over 2, 3000 tokens of 256: 94 and 109.  Heads of 64 need the registers for a
    // fourth wave: 8192 tokens, 16 over 4: 184 and 166.)
    constexpr bool kLate = DB > 64;
    __shared__ __attribute__((aligned(1024))) char ks[2][S * kTile];
    __shared__ __attribute__((aligned(1024))) char vs[2][S * kTile];
    __shared__ int dirty;
    // The longest rows first.  A (sequence, head) stays on one XCD, whose L2 then holds its
    // keys, where every XCD gets as many of each sequence; otherwise they go round.
    const unsigned heads = static_cast<unsigned>(a.heads_kv);
    int tile, head;
    Seq s;
    if (gathered) {
        head = static_cast<int>(blockIdx.x % heads);
        if (!gathered_tile(a, static_cast<int>(blockIdx.x / heads), s, tile)) return;
    } else {
        const unsigned per = static_cast<unsigned>(a.batch) * heads, turn = blockIdx.x / per;
        const unsigned which = heads % 8 == 0 ? blockIdx.x % per : (blockIdx.x + turn) % per;
        tile = static_cast<int>(tiles - 1 - turn);
        head = static_cast<int>(which % heads);
        s = sequence(a, static_cast<int>(which / heads));
    }
    const int rows = s.len_q * a.group;
    if (tile * 128 >= rows) return;
    const int stream = S == 1 ? 0 : static_cast<int>(wave_id() >> 2), wave = static_cast<int>(wave_id() & 3);
    const unsigned lane = threadIdx.x & 63;
    const int row0 = tile * 128 + wave * 32;

    const int sees = limit_of(a, s, tile * 128 + 127) + 1;       // keys any row of the workgroup sees
    const int free_to = limit_of(a, s, row0);                    // keys every row of the wave sees
    const int all = limit_of(a, s, tile * 128);                  // keys every row of the workgroup sees
    const bool hides = all < s.len_k - 1;
    const int n = sees > 0 ? (sees + KT - 1) / KT : 0;
    const int steps = (n + S - 1) / S;
    const int whole = min(steps, max(all + 1, 0) / KT / S);      // steps of tiles that every row sees whole
    const uint16_t *kp = static_cast<const uint16_t *>(a.k) + static_cast<size_t>(s.k0) * a.k_token +
                         static_cast<size_t>(head) * a.k_head;
    const uint16_t *vp = static_cast<const uint16_t *>(a.v) + static_cast<size_t>(s.k0) * a.v_token +
                         static_cast<size_t>(head) * a.v_head;
    Rows<T, DB> w;
    // In step u the keys of the next tile are loaded, and the values that the next step
    // multiplies.
    // Every pointer of a load into the next buffer and of a read of the present one is
    // restricted and none comes from a closure: only so does the compiler know that they
    // do not meet, and does not wait for the loads before the reads.
    typename Mat<T>::frag p[KT / 16];
    // the values of step u's tile, where some row does not see all of them
    const auto clean = [&](int u, char *vc) __attribute__((always_inline)) {
        if (!hides || u < whole) return;
        if (u * S + stream < n && clear_not_finite<T>(vc, kTile, static_cast<int>(threadIdx.x & 255), 256)) dirty = 1;
        __syncthreads();
    };
    auto general = [&](int u, bool start, const uint16_t *__restrict__ kg, const uint16_t *__restrict__ vg, char *__restrict__ kd,
                       char *__restrict__ vd, const char *__restrict__ kc, char *__restrict__ vc) __attribute__((always_inline)) {
        const int t = u * S + stream;
        if (start && t + S < n) {
            fill<DB, KT, 4, false>(kd, kg, a.k_token, (t + S) * KT, s.len_k, a.head_dim, wave);
            if (!kLate) fill<DB, KT, 4, true>(vd, vg, a.v_token, (t + S) * KT, s.len_k, a.head_dim, wave);
        }
        if (kLate && start && t < n) fill<DB, KT, 4, true>(vd, vg, a.v_token, t * KT, s.len_k, a.head_dim, wave);
        if (kLate && u > 0) {
            clean(u - 1, vc);
            if (t - S < n) tile_values<T, DB, KT>(vc, w, p);
        }
        if (!kLate) clean(u, vc);
        if (t < n) {
            tile_general<T, DB, KT>(kc, t * KT, free_to, a.scale_log2, w, p);
            if (!kLate) tile_values<T, DB, KT>(vc, w, p);
        }
    };
    // A tile that every row sees whole: its sums stay as they are unless a maximum has
    // outgrown its reference; then the tile is left to the general form.
    auto plain = [&](int u, const uint16_t *__restrict__ kg, const uint16_t *__restrict__ vg, char *__restrict__ kd,
                     char *__restrict__ vd, const char *__restrict__ kc, const char *__restrict__ vc)
                     __attribute__((always_inline)) -> bool {
        const int t = u * S + stream;
        if (t + S < n) {
            fill<DB, KT, 4, false>(kd, kg, a.k_token, (t + S) * KT, s.len_k, a.head_dim, wave);
            if (!kLate) fill<DB, KT, 4, true>(vd, vg, a.v_token, (t + S) * KT, s.len_k, a.head_dim, wave);
        }
        if (kLate) fill<DB, KT, 4, true>(vd, vg, a.v_token, t * KT, s.len_k, a.head_dim, wave);
        v16f sc[KT / 32];
        tile_scores<T, DB, KT>(kc, w, sc);
        const float top = tile_top<KT>(sc);
        if (__any(top * a.scale_log2 > w.m * a.scale_log2 + kSlack)) return false;
        if constexpr (kLate) {
            tile_both<T, DB, KT>(vc, sc, a.scale_log2, w, p);
        } else {
            tile_powers<T, DB, KT>(sc, a.scale_log2, w, p);
            tile_values<T, DB, KT>(vc, w, p);
        }
        return true;
    };
    if (threadIdx.x == 0) dirty = 0;
    const int mine = stream * kTile;
    if (stream < n) {
        fill<DB, KT, 4, false>(ks[0] + mine, kp, a.k_token, stream * KT, s.len_k, a.head_dim, wave);
        if (!kLate) fill<DB, KT, 4, true>(vs[0] + mine, vp, a.v_token, stream * KT, s.len_k, a.head_dim, wave);
    }
    start_rows<T, DB>(a, s, head, row0, w);
    int u = 0;
    bool begun = false;
    while (u < steps) {
        if (!begun) landed_for_all();   // the step's keys and values are there; everyone is done with the other buffers
        general(u, !begun, kp, vp, ks[(u + 1) & 1] + mine, vs[(u + 1 - kLate) & 1] + mine, ks[u & 1] + mine,
                vs[(u + kLate) & 1] + mine);
        begun = false;
        for (++u; u < whole; ++u) {
            landed_for_all();
            if (!plain(u, kp, vp, ks[(u + 1) & 1] + mine, vs[(u + 1 - kLate) & 1] + mine, ks[u & 1] + mine,
                       vs[(u + kLate) & 1] + mine)) {
                begun = true;
                break;
            }
        }
    }
    if (kLate && steps > 0) {
        landed_for_all();
        clean(steps - 1, vs[(steps - 1) & 1] + mine);
        if ((steps - 1) * S + stream < n) tile_values<T, DB, KT>(vs[(steps - 1) & 1] + mine, w, p);
    }
    if (hides && n > 0 && dirty != 0) {
        for (int t = whole * S + stream; t < n; t += S) {
            add_not_finite<T, DB>(vp, a.v_token, t * KT, min(t * KT + KT, sees), a.head_dim, w);
        }
    }

    float l = sum_halves(w.l);
    float mc = w.m == kNone ? kNone : w.m * a.scale_log2 - kLift<T>;
    if constexpr (S == 2) {   // the second stream's lanes hand theirs to the first's, lane by lane
        v4f *const sums = reinterpret_cast<v4f *>(ks);
        float *const stats = reinterpret_cast<float *>(vs);
        static_assert(DB / 8 * 256 * 16 <= static_cast<int>(sizeof(ks)), "the sums fit");
        const unsigned at = threadIdx.x & 255;
        __syncthreads();
        if (stream == 1) {
            stats[at] = mc;
            stats[256 + at] = l;
#pragma unroll
            for (int i = 0; i < DB / 32; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sums[(i * 4 + e) * 256 + at] = v4f{w.o[i][4 * e], w.o[i][4 * e + 1], w.o[i][4 * e + 2], w.o[i][4 * e + 3]};
                }
            }
        }
        __syncthreads();
        if (stream == 1) return;
        const float mc1 = stats[at], both = fmaxf(mc, mc1), base = both == kNone ? 0.0f : both;
        const float f0 = __builtin_amdgcn_exp2f(mc - base), f1 = __builtin_amdgcn_exp2f(mc1 - base);
        l = l * f0 + stats[256 + at] * f1;
        mc = both;
#pragma unroll
        for (int i = 0; i < DB / 32; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const v4f x = sums[(i * 4 + e) * 256 + at];
#pragma unroll
                for (int k = 0; k < 4; ++k) w.o[i][4 * e + k] = w.o[i][4 * e + k] * f0 + x[k] * f1;
            }
        }
    }
    const int r = row0 + static_cast<int>(lane & 31);
    if (r >= rows) return;
    const int token = r / a.group, sub = r - token * a.group;
    const size_t row = static_cast<size_t>(s.q0 + token);
    const int hq = head * a.group + sub;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const size_t at = row * a.o_token + static_cast<size_t>(hq) * a.o_head;
#pragma unroll
    for (int i = 0; i < DB / 32; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = i * 32 + e * 8 + static_cast<int>(lane >> 5) * 4;
            const float x[4] = {w.o[i][4 * e] * inv, w.o[i][4 * e + 1] * inv, w.o[i][4 * e + 2] * inv,
                                w.o[i][4 * e + 3] * inv};
            if (d < a.head_dim) store_n<T, 4>(a.out, at + d, x);
        }
    }
    if (a.lse != nullptr && lane < 32) {
        a.lse[row * a.heads_q + hq] = log_sum(mc == kNone ? 0.0f : mc, l);
    }
}

// Split calls keep (reference, sum) of every (row, split), then the weighted
// values of every (row, split).
LAYER_DEV float *part_sums(const AttnArgs &a) {
    const size_t stats = static_cast<size_t>(a.total_q) * a.heads_q * a.splits * 2;
    return a.part + ((stats + 3) & ~static_cast<size_t>(3));
}

// Part i of a call with several sequences, a part being 32 rows and a unit along the keys:
// all sequences' whole units first, then their last, shorter ones.  False past the last.  A
// lane counts every 64th sequence's.
LAYER_DEV bool gathered_part(const AttnArgs &a, int i, Seq &seq, int &part) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    const auto of = [&](int b) { return b < a.batch ? sequence(a, b) : Seq{0, 0, 0, 0}; };
    const Seq first = of(lane);
    for (int last = 0; last < 2; ++last) {
        for (int b = 0; b < a.batch; b += 64) {
            const Seq s = b == 0 ? first : of(b + lane);
            const int rows = s.len_q * a.group, keys = (max(limit_of(a, s, rows) + 1, 0) + 31) / 32, whole = keys / a.unit;
            const int tiles = (rows + 31) / 32, rest = keys > whole * a.unit || keys == 0 ? 1 : 0;
            const int n = tiles * (last == 0 ? whole : rest), to = sums_to(n);
            const unsigned long long past = __ballot(to > i);
            if (past != 0) {
                const int in = __ffsll(past) - 1;
                seq = lane_of(s, in);
                part = i + __builtin_amdgcn_readlane(n - to + (last == 0 ? 0 : tiles * whole), in);
                return true;
            }
            i -= __builtin_amdgcn_readlane(to, 63);
        }
    }
    return false;
}

// Few rows: the waves of a workgroup hold the same 32 rows and each takes every
// W-th tile of 32 keys of the workgroup's unit (a.unit tiles of the sequence), through
// LDS of its own, without a barrier until their sums are joined.  A wave has one buffer
// of keys and one of values: the next keys are under way while it multiplies
// the values, and the other way round.
// Bound by reading the keys and values: one token, 16 heads over 2 of 128, 131072 keys (134
// MB) take 27.3 us, 4.9 TB/s, and their join 6; 16 sequences of 1 to 4096 keys (93 MB) 25
// and 4.5.
template <int T, int DB, int W>
__global__ void __launch_bounds__(64 * W, DB <= 128 ? 2 : 1) k_attn_keys(AttnArgs a, unsigned tiles, bool gathered) {
    constexpr int KT = 32;
    constexpr int kTile = KT * DB * 2;
    constexpr int kPitch = DB + 4;
    constexpr int kSums = W * 16 * kPitch * 4;
    __shared__ __attribute__((aligned(1024))) char ks[kSums > W * kTile ? kSums : W * kTile];   // keys, later sums
    __shared__ __attribute__((aligned(1024))) char vs[W * kTile];
    __shared__ float stat[W][2][32];
    const unsigned heads = static_cast<unsigned>(a.heads_kv);
    const int head = static_cast<int>(blockIdx.x % heads);
    unsigned id = blockIdx.x / heads;
    int tile, unit;
    Seq s;
    if (gathered) {
        int part;
        if (!gathered_part(a, static_cast<int>(id), s, part)) return;
        const bool two = s.len_q * a.group > 32;      // (at most 64 rows)
        tile = two ? part % 2 : 0;
        unit = two ? part / 2 : part;
    } else {
        tile = static_cast<int>(id % tiles);
        id /= tiles;
        s = sequence(a, static_cast<int>(id % static_cast<unsigned>(a.batch)));
        unit = static_cast<int>(id / static_cast<unsigned>(a.batch));
    }
    const int rows = s.len_q * a.group, row0 = tile * 32;
    if (row0 >= rows) return;
    const int sees = limit_of(a, s, row0 + 31) + 1;
    const int n = sees > 0 ? (sees + KT - 1) / KT : 0;
    const int t0 = unit * a.unit, t1 = min(n, t0 + a.unit);
    if (t0 >= n && unit > 0) return;          // (the first unit also answers for rows that see nothing)
    const bool alone = n <= a.unit;                 // no other unit of these rows
    const int wave = static_cast<int>(wave_id());
    const unsigned lane = threadIdx.x & 63;

    const int free_to = limit_of(a, s, row0);
    const uint16_t *kp = static_cast<const uint16_t *>(a.k) + static_cast<size_t>(s.k0) * a.k_token +
                         static_cast<size_t>(head) * a.k_head;
    const uint16_t *vp = static_cast<const uint16_t *>(a.v) + static_cast<size_t>(s.k0) * a.v_token +
                         static_cast<size_t>(head) * a.v_head;
    char *const kw = ks + wave * kTile, *const vw = vs + wave * kTile;
    if (t0 + wave < t1) {
        fill<DB, KT, 1, false, true>(kw, kp, a.k_token, (t0 + wave) * KT, s.len_k, a.head_dim, 0);
        fill<DB, KT, 1, true, true>(vw, vp, a.v_token, (t0 + wave) * KT, s.len_k, a.head_dim, 0);
    }
    Rows<T, DB> w;
    start_rows<T, DB>(a, s, head, row0, w);
    const bool hides = free_to < s.len_k - 1;
    bool dirty = false;
    landed_for_wave();
    typename Mat<T>::frag p[KT / 16];
    // (restricted pointers, as in the kernel above)
    auto values = [&](int t, const uint16_t *__restrict__ kg, char *__restrict__ kd, char *__restrict__ vc)
                      __attribute__((always_inline)) {
        if (t + W < t1) {
            read_by_wave();                         // before the keys' buffer is filled again
            fill<DB, KT, 1, false>(kd, kg, a.k_token, (t + W) * KT, s.len_k, a.head_dim, 0);
            landed_but<DB / 16>();                  // the values; the next keys are under way
        } else {
            landed_for_wave();
        }
        if (hides && t * KT + KT - 1 > free_to && clear_not_finite<T>(vc, kTile, static_cast<int>(lane), 64)) dirty = true;
        tile_values<T, DB, KT>(vc, w, p);
    };
    for (int t = t0 + wave; t < t1; t += W) {
        if (t != t0 + wave) landed_but<DB / 16>();  // the keys; the values may be under way
        tile_general<T, DB, KT>(kw, t * KT, free_to, a.scale_log2, w, p);
        values(t, kp, kw, vw);
        if (t + W < t1) {
            read_by_wave();                         // before the values' is
            fill<DB, KT, 1, true>(vw, vp, a.v_token, (t + W) * KT, s.len_k, a.head_dim, 0);
        }
    }
    if (__any(dirty)) {
        for (int t = t0 + wave; t < t1; t += W) {
            if (t * KT + KT - 1 > free_to) {
                add_not_finite<T, DB>(vp, a.v_token, t * KT, min(t * KT + KT, sees), a.head_dim, w);
            }
        }
    }

    // join the waves: each scales its sums to the common reference
    const float mc_own = w.m == kNone ? kNone : w.m * a.scale_log2 - kLift<T>;
    const float l_own = sum_halves(w.l);
    if (lane < 32) {
        stat[wave][0][lane] = mc_own;
        stat[wave][1][lane] = l_own;
    }
    __syncthreads();
    const unsigned col = lane & 31;
    float mc = kNone;
#pragma unroll
    for (int i = 0; i < W; ++i) mc = fmaxf(mc, stat[i][0][col]);
    const float own = __builtin_amdgcn_exp2f(mc_own - (mc == kNone ? 0.0f : mc));
    float *const sums = reinterpret_cast<float *>(ks);   // [wave][row][kPitch]
#pragma unroll
    for (int half = 0; half < 2; ++half) {          // 16 rows at a time fit there
        if (static_cast<int>(col >> 4) == half) {
#pragma unroll
            for (int i = 0; i < DB / 32; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = i * 32 + e * 8 + static_cast<int>(lane >> 5) * 4;
                    const v4f x = {w.o[i][4 * e] * own, w.o[i][4 * e + 1] * own, w.o[i][4 * e + 2] * own,
                                   w.o[i][4 * e + 3] * own};
                    *reinterpret_cast<v4f *>(sums + (wave * 16 + (col & 15)) * kPitch + d) = x;
                }
            }
        }
        __syncthreads();
        // all threads: four elements of a row each
        constexpr int kQuads = DB / 4;
        for (int i = static_cast<int>(threadIdx.x); i < 16 * kQuads; i += 64 * W) {
            const int c = i / kQuads, d = (i - c * kQuads) * 4, r = row0 + half * 16 + c;
            if (r >= rows || d >= a.head_dim) continue;
            v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
            float top = kNone, total = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const v4f y = *reinterpret_cast<const v4f *>(sums + (k * 16 + c) * kPitch + d);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] += y[e];
                top = fmaxf(top, stat[k][0][half * 16 + c]);
            }
            const float base = top == kNone ? 0.0f : top;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                total += stat[k][1][half * 16 + c] * __builtin_amdgcn_exp2f(stat[k][0][half * 16 + c] - base);
            }
            const int token = r / a.group, sub = r - token * a.group;
            const size_t row = static_cast<size_t>(s.q0 + token);
            const int hq = head * a.group + sub;
            if (alone) {
                const float inv = total == 0.0f ? 0.0f : 1.0f / total;
                const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
                store_n<T, 4>(a.out, row * a.o_token + static_cast<size_t>(hq) * a.o_head + d, y);
                if (a.lse != nullptr && d == 0) a.lse[row * a.heads_q + hq] = log_sum(base, total);
            } else {
                const size_t entry = (row * a.heads_q + hq) * a.splits + unit;
                *reinterpret_cast<v4f *>(part_sums(a) + entry * a.head_dim + d) = x;
                if (d == 0) {
                    a.part[entry * 2] = top;
                    a.part[entry * 2 + 1] = total;
                }
            }
        }
        __syncthreads();
    }
}

// Joins the units of a row: a workgroup for each (query, head).  Lane groups take every
// G-th unit's sums, which are then added in the order of the groups.
template <int T>
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs a) {
    __shared__ float weight[256], top_of[4], total_of[4];
    __shared__ v4f part[256];
    const int thread = static_cast<int>(threadIdx.x);
    const int hq = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.heads_q));
    const int token = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.heads_q));
    const Seq s = sequence(a, static_cast<int>(blockIdx.y));
    if (token >= s.len_q) return;
    // the units this row's workgroups made: those of the last row of its 32
    const int row32 = (token * a.group + hq % a.group) / 32 * 32;
    const int sees = limit_of(a, s, row32 + 31) + 1;
    const int tiles = sees > 0 ? (sees + 31) / 32 : 0, n = (tiles + a.unit - 1) / a.unit;
    if (n <= 1) return;                             // written whole
    const size_t row = static_cast<size_t>(s.q0 + token);
    const size_t entry = (row * a.heads_q + hq) * a.splits;
    const float *stats = a.part + entry * 2;
    const float *sums = part_sums(a) + entry * a.head_dim;

    const float mine = thread < n ? stats[2 * thread] : kNone;
    float top = mine;
    for (int step = 1; step < 64; step <<= 1) top = fmaxf(top, __shfl_xor(top, step));
    if ((thread & 63) == 0) top_of[thread >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(top_of[0], top_of[1]), fmaxf(top_of[2], top_of[3]));
    const float base = top == kNone ? 0.0f : top;
    const float f = thread < n ? __builtin_amdgcn_exp2f(mine - base) : 0.0f;
    weight[thread] = f;
    float total = thread < n ? stats[2 * thread + 1] * f : 0.0f;
    for (int step = 1; step < 64; step <<= 1) total += __shfl_xor(total, step);
    if ((thread & 63) == 0) total_of[thread >> 6] = total;
    __syncthreads();
    total = (total_of[0] + total_of[1]) + (total_of[2] + total_of[3]);

    const int quads = a.head_dim / 4, groups = 256 / quads;
    const int group = thread / quads, d = (thread - group * quads) * 4;
    v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (group < groups) {
        // eight loads under way at a time, added in order
        constexpr int kAhead = 8;
        for (int i = group; i < n; i += groups * kAhead) {
            v4f y[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int at = i + k * groups;
                y[k] = *reinterpret_cast<const v4f *>(sums + static_cast<size_t>(at < n ? at : i) * a.head_dim + d);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int at = i + k * groups;
                const float scale = at < n ? weight[at] : 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = at < n ? __builtin_fmaf(y[k][e], scale, x[e]) : x[e];
            }
        }
        part[thread] = x;
    }
    __syncthreads();
    if (group != 0) return;
    const int used = groups < n ? groups : n;
    for (int i = 1; i < used; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += part[i * quads + thread][e];
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
    store_n<T, 4>(a.out, row * a.o_token + static_cast<size_t>(hq) * a.o_head + d, y);
    if (a.lse != nullptr && thread == 0) a.lse[row * a.heads_q + hq] = log_sum(base, total);
}

template <int T, int DB>
hipError_t launch_dim(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    const unsigned rows = static_cast<unsigned>(a.max_q) * static_cast<unsigned>(a.group);
    if (!p.split) {
        const unsigned tiles = (rows + 127) / 128;
        const dim3 grid(static_cast<unsigned>(p.tiles) * static_cast<unsigned>(a.heads_kv));
        if constexpr (DB <= 128) {
            if (p.streams == 2) {
                hipLaunchKernelGGL((k_attn_rows<T, DB, 2>), grid, dim3(512), 0, stream, a, tiles, p.gathered);
                return hipGetLastError();
            }
        }
        hipLaunchKernelGGL((k_attn_rows<T, DB, 1>), grid, dim3(256), 0, stream, a, tiles, p.gathered);
        return hipGetLastError();
    }
    const unsigned tiles = (rows + 31) / 32, per = static_cast<unsigned>(a.batch * a.heads_kv);
    hipLaunchKernelGGL((k_attn_keys<T, DB, 4>), dim3(tiles * per * static_cast<unsigned>(p.splits)), dim3(256), 0, stream, a, tiles, p.gathered);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    hipLaunchKernelGGL((k_attn_join<T>), dim3(static_cast<unsigned>(a.max_q) * static_cast<unsigned>(a.heads_q),
                                              static_cast<unsigned>(a.batch)),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <int T>
hipError_t launch_t(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    if (a.head_dim <= 64) return launch_dim<T, 64>(a, p, stream);
    if (a.head_dim <= 128) return launch_dim<T, 128>(a, p, stream);
    return launch_dim<T, 256>(a, p, stream);
}

}  // namespace

AttnPlan plan_attn(const ar_attn &s) {
    AttnPlan p{};
    p.splits = 1;
    const size_t rows = static_cast<size_t>(s.max_q) * static_cast<size_t>(s.heads_q / s.heads_kv);
    p.split = rows <= 64;
    if (!p.split) {
        // Tiles with work, at most: counted by rows, each sequence's last one may be part
        // empty; or by the longest sequence, which needs no search for a workgroup's tile but
        // starts empty ones where lengths differ (ten of 10 tokens, six of 30 to 3000,
        // 32 heads over 8 of 128: 137 us gathered, 263 not).
        const size_t group = static_cast<size_t>(s.heads_q / s.heads_kv), batch = static_cast<size_t>(s.batch);
        const size_t by_rows = (s.total_q * group + 127) / 128 + batch, by_length = (rows + 127) / 128 * batch;
        p.gathered = by_rows < by_length;
        p.tiles = std::min(by_rows, by_length);
        // Two streams halve the longest rows' time, one keeps more workgroups of different
        // progress on a CU.  (us on MI355X, two streams and one; 32 heads over 8, causal.)
        // head_dim 128, where a CU holds one workgroup of two streams: up to one for each CU
        // (1024 tokens: 24 and 26.5), up to twice that where one sequence has most of them and
        // its rows differ in length (1300 tokens: 33 and 36, 16 heads over 4, 4000: 81 and 91; not
        // for two of 1000: 35 and 32, nor where all rows are long, 1200 tokens over 9000 keys: 239
        // and 222; 4096 tokens: 163 and 158).
        // head_dim 64, where it holds two: up to that (1200 tokens, 9000 keys: 135 and 150), up to
        // twice that where the longest are 32 steps (16 over 4, 5000 tokens: 77 and 89; three
        // times 1000 tokens: 29 and 26).
        const size_t wgs = p.tiles * static_cast<size_t>(s.heads_kv);
        const size_t keys = longest_keys(s), tokens = static_cast<size_t>(s.max_q);
        const bool two = s.head_dim <= 64    ? wgs <= 512 || (wgs <= 1024 && keys > 31 * 64)
                         : s.head_dim <= 128 ? wgs <= 256 || (wgs <= 512 && keys < 2 * tokens && (rows + 127) / 128 * 2 > p.tiles)
                                             : false;
        p.streams = two ? 2 : 1;
        return p;
    }
    const size_t wgs = ((rows + 31) / 32) * static_cast<size_t>(s.batch) * static_cast<size_t>(s.heads_kv);
    const size_t tiles = (longest_keys(s) + 31) / 32;
    // Units of whole rounds of the four waves: about ten for each CU, so that
    // sequences of different lengths even out, but none under two rounds.  (us with ten, six and
    // three; 8 key heads: 63 sequences of 10 keys and one of 8000: 27, 35, 46; 32 of 2000: 62, 60,
    // 58; 100 of 1 to 4000: 172, 172, 170.)
    size_t unit = (wgs * tiles + 2559) / 2560;
    if (unit < (tiles + 255) / 256) unit = (tiles + 255) / 256;
    unit = (unit + 3) / 4 * 4;
    if (unit < 8) unit = 8;
    const size_t splits = tiles > unit ? (tiles + unit - 1) / unit : 1;
    // Gathered where the call has more workgroups than the chip holds at once, two on a CU: those
    // that end at once, between the others, take CUs' turns in the dispatch (16 sequences of 1
    // to 4096 keys, 8 key heads: 27 us gathered, 29.6 not).
    p.gathered = s.batch > 1 && wgs * splits > 512;
    p.unit = static_cast<int>(unit);
    p.splits = static_cast<int>(splits);
    if (splits > 1) {
        const size_t entries = s.total_q * static_cast<size_t>(s.heads_q) * splits;
        p.workspace = ((entries * 2 + 3) / 4 * 4 + entries * static_cast<size_t>(s.head_dim)) * 4;
    }
    return p;
}

hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, ar_dtype type, hipStream_t stream) {
    return type == AR_F16 ? launch_t<AR_F16>(a, p, stream) : launch_t<AR_BF16>(a, p, stream);
}

}  // namespace layer
}  // namespace mpp

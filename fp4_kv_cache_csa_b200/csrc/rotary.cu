// rotary.cu -- rotary positions: every pair of channels (a, b) of a vector is
// turned by an angle that grows with the vector's token position,
//
//   y_a = s (a cos t - b sin t),   y_b = s (a sin t + b cos t),   t = pos * f_p
//
// (the inverse turns by -t). Entries of a compressed cache are key and value at
// once, so a caller rotates queries, tokens and window rows on their way in and
// turns attention outputs back with the inverse. The map is linear and its
// transpose is the inverse with the same s, so the inverse is also the gradient.
//
// Angles: pos has 31 bits and f_p 24, so the float64 product is exact to 2^-53
// relative, and it is reduced to [-pi, pi] in float64 with 2 pi in two parts
// (an argument of 2^20 would lose all but four bits of its fraction in float32);
// sine and cosine of the reduced angle, taken as a multiple of pi, are float32.
//
// HBM-bound: each vector is read and written once (in place only its rotated
// channels). One CTA takes a run of vectors (token, head), about four 8-channel
// chunks per thread, all loaded before the angles are computed, so that the
// table of the run's cosines and sines (one entry per token and pair, shared by
// the token's heads) is built while the loads are in flight.
#include <cuda_bf16.h>

#include "common.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kUnitsPerThread = 4;
constexpr int kTable = 4096;  // (token, pair) entries of the table, 32 KB; one token's pairs always fit (dim <= 8192)

struct RotaryArgs {
    const void *x;
    void *out;
    const int32_t *pos;
    const float *inv_freq;
    long long x_row, x_head, out_row, out_head;  // strides in elements
    long long vectors;                           // rows * heads
    int heads, dim, rot_begin, rot_dim, half;
    int units;       // work units of a vector: copied ones first, then rotated ones
    int copy_units;  // 0 in place
    int per_cta;     // vectors of a CTA
    float mscale, sign;
};

// ch consecutive channels, as the 32-bit words that hold them
template <typename T, int CH>
struct Words {
    static constexpr int N = (CH * (int)sizeof(T) + 3) / 4;
    uint32_t w[N];
};

template <typename T, int CH>
__device__ __forceinline__ Words<T, CH> load(const T *p) {
    Words<T, CH> r;
    if constexpr (CH * sizeof(T) >= 16) {
#pragma unroll
        for (int k = 0; k < (int)(CH * sizeof(T)) / 16; ++k) {
            const uint4 u = reinterpret_cast<const uint4 *>(p)[k];
            r.w[4 * k] = u.x;
            r.w[4 * k + 1] = u.y;
            r.w[4 * k + 2] = u.z;
            r.w[4 * k + 3] = u.w;
        }
    } else if constexpr (sizeof(T) == 4) {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        r.w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
    return r;
}

template <typename T, int CH>
__device__ __forceinline__ void unpack(const Words<T, CH> &r, float (&v)[CH]) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        if constexpr (sizeof(T) == 4) v[k] = __uint_as_float(r.w[k]);
        else v[k] = __uint_as_float((k & 1) ? (r.w[k >> 1] & 0xFFFF0000u) : (r.w[k >> 1] << 16));
    }
}

// Stores round once, to the output's type (bf16: to nearest even).
template <typename T, int CH>
__device__ __forceinline__ void store(T *p, const float (&v)[CH]) {
    if constexpr (CH == 1) {
        if constexpr (sizeof(T) == 4) *p = v[0];
        else *p = __float2bfloat16_rn(v[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < CH; k += 4)
            reinterpret_cast<float4 *>(p)[k / 4] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    } else {
        uint32_t w[CH / 2];
#pragma unroll
        for (int k = 0; k < CH; k += 2) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[k], v[k + 1]);
            w[k / 2] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// pos * f reduced to [-pi, pi], then (cos, sin) * mscale
__device__ __forceinline__ float2 angle(int pos, float f, float mscale, float sign) {
    constexpr double kInvPi = 0.31830988618379067154;
    constexpr double kInv2Pi = 0.15915494309189533577;
    constexpr double kTwoPiHi = 6.28318530717958623200;   // 2 pi rounded to float64 ...
    constexpr double kTwoPiLo = 2.44929359829470635e-16;  // ... and what it lacks
    const double t = (double)pos * (double)f;
    const double k = rint(t * kInv2Pi);
    const double r = fma(-k, kTwoPiLo, fma(-k, kTwoPiHi, t));
    float s, c;
    sincospif((float)(r * kInvPi), &s, &c);
    return make_float2(c * mscale, s * mscale * sign);
}

// CH = 8: chunks of 16 or 32 bytes; CH = 1: one channel (or pair) at a time, for
// vectors whose addresses or rotated range do not fall on 16-byte boundaries.
template <typename TI, typename TO, int CH>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a) {
    __shared__ float2 table[kTable];
    const long long v0 = (long long)blockIdx.x * a.per_cta;
    const int nv = (int)min((long long)a.per_cta, a.vectors - v0);
    const long long row0 = v0 / a.heads;
    const int head0 = (int)(v0 - row0 * a.heads);
    const int pairs = a.rot_dim >> 1;
    const TI *x = static_cast<const TI *>(a.x);
    TO *out = static_cast<TO *>(a.out);
    // a vector with more units than a CTA takes is spread over blockIdx.y (then per_cta is 1)
    const unsigned units = a.units, u_first = blockIdx.y * (kThreads * kUnitsPerThread);
    const unsigned total = (unsigned)nv * units;

    // channels of a unit: c0, and c1 (the partners, CH channels further on, or the pair's second channel)
    struct Unit {
        long long xo, oo;
        int c0, c1, p, rl;  // first channels, first pair, row of the run; p < 0: copied
    };
    auto locate = [&](unsigned u) {
        Unit r;
        const unsigned lv = u / units, k = u - lv * units;
        const unsigned hh = (unsigned)head0 + lv;
        r.rl = (int)(hh / (unsigned)a.heads);
        const long long row = row0 + r.rl;
        const int head = (int)(hh - (unsigned)r.rl * (unsigned)a.heads);
        r.xo = row * a.x_row + head * a.x_head;
        r.oo = row * a.out_row + head * a.out_head;
        if ((int)k < a.copy_units) {
            r.c0 = (int)k * CH;
            if (r.c0 >= a.rot_begin) r.c0 += a.rot_dim;  // the channels behind the rotated ones
            r.c1 = -1;
            r.p = -1;
        } else {
            const int j = (int)k - a.copy_units;
            if (a.half) {
                r.p = j * CH;
                r.c0 = a.rot_begin + r.p;
                r.c1 = r.c0 + pairs;
            } else if constexpr (CH == 1) {
                r.p = j;
                r.c0 = a.rot_begin + 2 * j;
                r.c1 = r.c0 + 1;
            } else {
                r.p = j * (CH / 2);
                r.c0 = a.rot_begin + j * CH;
                r.c1 = -1;
            }
        }
        return r;
    };

    Words<TI, CH> w0[kUnitsPerThread], w1[kUnitsPerThread];
#pragma unroll
    for (int i = 0; i < kUnitsPerThread; ++i) {
        const unsigned u = u_first + threadIdx.x + i * kThreads;
        if (u < total) {
            const Unit r = locate(u);
            w0[i] = load<TI, CH>(x + r.xo + r.c0);
            if (r.c1 >= 0) w1[i] = load<TI, CH>(x + r.xo + r.c1);
        }
    }
    const int nrows = nv > 0 ? (head0 + nv - 1) / a.heads + 1 : 0;
    for (int k = threadIdx.x; k < nrows * pairs; k += kThreads) {
        const int rl = k / pairs, p = k - rl * pairs;
        table[k] = angle(__ldg(a.pos + row0 + rl), __ldg(a.inv_freq + p), a.mscale, a.sign);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kUnitsPerThread; ++i) {
        const unsigned u = u_first + threadIdx.x + i * kThreads;
        if (u >= total) break;
        const Unit r = locate(u);
        float v[CH];
        unpack<TI, CH>(w0[i], v);
        if (r.p < 0) {
            store<TO, CH>(out + r.oo + r.c0, v);
            continue;
        }
        const float2 *cs = table + r.rl * pairs + r.p;
        if (r.c1 >= 0) {
            float b[CH];
            unpack<TI, CH>(w1[i], b);
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const float2 t = cs[k];
                const float y = v[k] * t.x - b[k] * t.y;
                b[k] = v[k] * t.y + b[k] * t.x;
                v[k] = y;
            }
            store<TO, CH>(out + r.oo + r.c0, v);
            store<TO, CH>(out + r.oo + r.c1, b);
        } else if constexpr (CH > 1) {
#pragma unroll
            for (int k = 0; k < CH; k += 2) {
                const float2 t = cs[k / 2];
                const float y = v[k] * t.x - v[k + 1] * t.y;
                v[k + 1] = v[k] * t.y + v[k + 1] * t.x;
                v[k] = y;
            }
            store<TO, CH>(out + r.oo + r.c0, v);
        }
    }
}

template <typename TI, typename TO, int CH>
cudaError_t launch(RotaryArgs a, bool in_place, cudaStream_t s) {
    a.copy_units = in_place ? 0 : (a.dim - a.rot_dim) / CH;
    a.units = a.copy_units + ((a.half || CH == 1) ? a.rot_dim / 2 / CH : a.rot_dim / CH);
    const int by_units = kThreads * kUnitsPerThread / a.units;
    const int by_table = kTable / (a.rot_dim / 2);
    a.per_cta = max(1, min(by_units, by_table));
    const long long grid = (a.vectors + a.per_cta - 1) / a.per_cta;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int slices = a.per_cta > 1 ? 1 : (a.units + kThreads * kUnitsPerThread - 1) / (kThreads * kUnitsPerThread);
    rotary_kernel<TI, TO, CH><<<dim3((unsigned)grid, slices), dim3(kThreads), 0, s>>>(a);
    return cudaGetLastError();
}

template <typename TI, typename TO>
cudaError_t launch_types(const RotaryArgs &a, bool vec, bool in_place, cudaStream_t s) {
    return vec ? launch<TI, TO, 8>(a, in_place, s) : launch<TI, TO, 1>(a, in_place, s);
}

}  // namespace

cudaError_t launch_rotary(const csa_vectors &x, const csa_vectors &out, int rows, int heads, int dim,
                          const csa_rope &rope, const int32_t *pos, bool inverse, bool in_place, cudaStream_t s) {
    RotaryArgs a = {};
    a.x = x.data;
    a.out = out.data;
    a.pos = pos;
    a.inv_freq = rope.inv_freq;
    a.x_row = x.row_stride;
    a.x_head = x.head_stride;
    a.out_row = out.row_stride;
    a.out_head = out.head_stride;
    a.vectors = (long long)rows * heads;
    a.heads = heads;
    a.dim = dim;
    a.rot_begin = rope.rot_begin;
    a.rot_dim = rope.rot_dim;
    a.half = rope.layout == CSA_ROPE_HALF;
    a.mscale = rope.mscale;
    a.sign = inverse ? -1.f : 1.f;
    // 8-channel chunks: the rotated range starts and ends on a chunk (half layout: both of its
    // halves do), and every vector starts on 16 bytes in both tensors
    auto aligned = [&](const csa_vectors &v) {
        const long long per16 = v.dtype == CSA_BF16 ? 8 : 4;
        return reinterpret_cast<uintptr_t>(v.data) % 16 == 0 && (rows == 1 || v.row_stride % per16 == 0) &&
               (heads == 1 || v.head_stride % per16 == 0);
    };
    const bool vec = dim % 8 == 0 && rope.rot_begin % 8 == 0 && rope.rot_dim % (a.half ? 16 : 8) == 0 && aligned(x) &&
                     aligned(out);
    if (x.dtype == CSA_BF16)
        return out.dtype == CSA_BF16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(a, vec, in_place, s)
                                     : launch_types<__nv_bfloat16, float>(a, vec, in_place, s);
    return out.dtype == CSA_BF16 ? launch_types<float, __nv_bfloat16>(a, vec, in_place, s)
                                 : launch_types<float, float>(a, vec, in_place, s);
}

}  // namespace csa

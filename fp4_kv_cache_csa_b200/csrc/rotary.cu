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
// sine and cosine of the reduced angle, taken as a multiple of pi, are float32, and turned on by what that
// multiple's rounding left (without it float32 outputs are 1.2 to 1.5 times as far from the exact ones).
//
// HBM-bound: each vector is read and written once (in place only its rotated
// channels). A CTA takes a run of vectors (token, head), about four 8-channel
// chunks per thread, and either their rotated channels or the copied ones. The
// former are loaded before the angles are computed, so that the table of the
// run's cosines and sines (one entry per token and pair, shared by the token's
// heads) is built while the loads are in flight; copies have nothing to wait for
// (both in one CTA: 210 us for 8192 x 64 x 512 bf16, apart: 175 us; in place, 64 channels
// of each vector, 29 us against 20 of the bytes). Vectors off 16 bytes go one channel at a
// time: 690 us, in place 81.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
// chunks of a thread: four of bf16, two of float32 (a pair of chunks in half layout: 64 registers at four, and two
// CTAs an SM)
template <typename T>
constexpr int units_per_thread() { return sizeof(T) == 4 ? 2 : 4; }
constexpr int kTable = 4096;  // (token, pair) entries of the table, 32 KB; one token's pairs always fit (dim <= 8192)

struct RotaryArgs {
    const void *x;
    void *out;
    const int32_t *pos;
    const float *inv_freq;
    long long x_row, x_head, out_row, out_head;  // strides in elements
    long long vectors;                           // rows * heads
    int heads, dim, rot_begin, rot_dim, half;
    // [0] rotated channels, [1] copied ones: work units of a vector, and its quotient's factor (see quotient()),
    // vectors of a CTA, CTAs
    int units[2], per_cta[2];
    uint32_t units_rcp[2], heads_rcp;
    unsigned ctas[2];
    float mscale, sign;
    bool wide_x, wide_out;
};

// n / d from rcp = 2^32 / d + 1, exact for n d < 2^32: here n < 2^16 and d < 2^15. (d = 1: rcp = 0.) Two divisions a
// unit were most of its instructions: 246 -> 210 us for 8192 x 64 x 512 bf16.
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t rcp) { return rcp ? __umulhi(n, rcp) : n; }
constexpr int kManyHeads = 1 << 15;  // from here on a run of vectors meets at most one row's end

// ch consecutive channels, as the 32-bit words that hold them
template <typename T, int CH>
struct Words {
    static constexpr int N = (CH * (int)sizeof(T) + 3) / 4;
    uint32_t w[N];
};

// wide: p lies on a 32-byte boundary, and eight float32 go in one access (two of 16 bytes, each a half of every lane's
// sector, take the L1 twice as long).
template <typename T, int CH>
__device__ __forceinline__ Words<T, CH> load(const T *p, bool wide) {
    Words<T, CH> r;
    if (CH * sizeof(T) == 32 && wide) {
        if constexpr (CH * sizeof(T) == 32)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                           "=r"(r.w[7])
                         : "l"(p)
                         : "memory");
    } else if constexpr (CH * sizeof(T) >= 16) {
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
__device__ __forceinline__ void store(T *p, const float (&v)[CH], bool wide) {
    if (CH * sizeof(T) == 32 && wide) {
        if constexpr (CH * sizeof(T) == 32)
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                         "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                         : "memory");
    } else if constexpr (CH == 1) {
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

// The words of channels that keep their type, as they are (a conversion would rewrite the payloads of NaNs).
template <typename T, int CH>
__device__ __forceinline__ void store_words(T *p, const Words<T, CH> &r, bool wide) {
    if (CH * sizeof(T) == 32 && wide) {
        if constexpr (CH * sizeof(T) == 32)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]),
                         "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
                         : "memory");
    } else if constexpr (CH * sizeof(T) >= 16) {
#pragma unroll
        for (int k = 0; k < (int)(CH * sizeof(T)) / 16; ++k)
            reinterpret_cast<uint4 *>(p)[k] = make_uint4(r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<uint32_t *>(p) = r.w[0];
    } else {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)r.w[0];
    }
}

// pos * f reduced to [-pi, pi], then (cos, sin) * mscale
__device__ __forceinline__ float2 angle(int pos, float f, float mscale, float sign) {
    constexpr double kPi = 3.14159265358979311600, kInvPi = 0.31830988618379067154;
    constexpr double kInv2Pi = 0.15915494309189533577;
    constexpr double kTwoPiHi = 6.28318530717958623200;   // 2 pi rounded to float64 ...
    constexpr double kTwoPiLo = 2.44929359829470635e-16;  // ... and what it lacks
    const double t = (double)pos * (double)f;
    const double k = rint(t * kInv2Pi);
    const double r = fma(-k, kTwoPiLo, fma(-k, kTwoPiHi, t));
    float s, c;
    const float turns = (float)(r * kInvPi);
    sincospif(turns, &s, &c);
    const float rest = (float)fma(-kPi, (double)turns, r);  // what turns' rounding left of the angle, up to 2^-23
    return make_float2(fmaf(-s, rest, c) * mscale, fmaf(c, rest, s) * mscale * sign);
}

// CH = 8: chunks of 16 or 32 bytes; CH = 1: one channel (or pair) at a time, for
// vectors whose addresses or rotated range do not fall on 16-byte boundaries.
template <typename TI, typename TO, int CH>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a) {
    constexpr int UPT = units_per_thread<TI>();
    extern __shared__ float2 table[];  // [rows of the run][pairs]
    const int copies = blockIdx.x >= a.ctas[0];
    const unsigned block = blockIdx.x - (copies ? a.ctas[0] : 0);
    const int units = a.units[copies], per_cta = a.per_cta[copies];
    // a vector with more units than a CTA takes is spread over blockIdx.y (then per_cta is 1)
    const unsigned u_first = blockIdx.y * (kThreads * UPT);
    const long long v0 = (long long)block * per_cta;
    const int nv = (int)min((long long)per_cta, a.vectors - v0);
    const unsigned total = (unsigned)nv * units;
    if (u_first >= total) return;
    const long long row0 = v0 / a.heads;
    const int head0 = (int)(v0 - row0 * a.heads);
    const TI *x = static_cast<const TI *>(a.x) + row0 * a.x_row;
    TO *out = static_cast<TO *>(a.out) + row0 * a.out_row;
    const uint32_t rcp = a.units_rcp[copies];

    // the vector of a unit (its row of the run, its offsets), and the unit's number in it
    struct Unit {
        long long xo, oo;
        int k, rl;
    };
    auto locate = [&](unsigned u) {
        Unit r;
        const unsigned lv = quotient(u, rcp), hh = (unsigned)head0 + lv;
        r.k = (int)(u - lv * units);
        r.rl = a.heads >= kManyHeads ? hh >= (unsigned)a.heads : (int)quotient(hh, a.heads_rcp);
        const int head = (int)(hh - (unsigned)r.rl * (unsigned)a.heads);
        r.xo = r.rl * a.x_row + head * a.x_head;
        r.oo = r.rl * a.out_row + head * a.out_head;
        return r;
    };

    if (copies) {
        Words<TI, CH> w[UPT];
        long long to[UPT];
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const unsigned u = u_first + threadIdx.x + i * kThreads;
            if (u < total) {
                const Unit r = locate(u);
                int c = r.k * CH;
                if (c >= a.rot_begin) c += a.rot_dim;  // the channels behind the rotated ones
                w[i] = load<TI, CH>(x + r.xo + c, a.wide_x);
                to[i] = r.oo + c;
            }
        }
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            if (u_first + threadIdx.x + i * kThreads >= total) break;
            if constexpr (std::is_same<TI, TO>::value) {
                store_words<TO, CH>(out + to[i], w[i], a.wide_out);
            } else {
                float v[CH];
                unpack<TI, CH>(w[i], v);
                store<TO, CH>(out + to[i], v, a.wide_out);
            }
        }
        return;
    }

    const int pairs = a.rot_dim >> 1;
    // channels of a unit: c0, and its partners' c1 (-1: they are in the same chunk); p: its first pair
    auto channels = [&](int k, int &c0, int &c1, int &p) {
        p = a.half || CH == 1 ? k * CH : k * (CH / 2);
        c0 = a.rot_begin + (a.half ? p : 2 * p);
        c1 = a.half ? c0 + pairs : CH == 1 ? c0 + 1 : -1;
    };
    Words<TI, CH> w0[UPT], w1[UPT];
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
        const unsigned u = u_first + threadIdx.x + i * kThreads;
        if (u < total) {
            const Unit r = locate(u);
            int c0, c1, p;
            channels(r.k, c0, c1, p);
            w0[i] = load<TI, CH>(x + r.xo + c0, a.wide_x);
            if (c1 >= 0) w1[i] = load<TI, CH>(x + r.xo + c1, a.wide_x);
        }
    }
    const int nrows = (head0 + nv - 1) / a.heads + 1;
    for (int k = threadIdx.x; k < nrows * pairs; k += kThreads) {
        const int rl = k / pairs, p = k - rl * pairs;
        table[k] = angle(__ldg(a.pos + row0 + rl), __ldg(a.inv_freq + p), a.mscale, a.sign);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
        const unsigned u = u_first + threadIdx.x + i * kThreads;
        if (u >= total) break;
        const Unit r = locate(u);
        int c0, c1, p;
        channels(r.k, c0, c1, p);
        float v[CH];
        unpack<TI, CH>(w0[i], v);
        const float2 *cs = table + r.rl * pairs + p;
        if (c1 >= 0) {
            float b[CH];
            unpack<TI, CH>(w1[i], b);
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const float2 t = cs[k];
                const float y = v[k] * t.x - b[k] * t.y;
                b[k] = v[k] * t.y + b[k] * t.x;
                v[k] = y;
            }
            store<TO, CH>(out + r.oo + c0, v, a.wide_out);
            store<TO, CH>(out + r.oo + c1, b, a.wide_out);
        } else if constexpr (CH > 1) {
#pragma unroll
            for (int k = 0; k < CH; k += 2) {
                const float2 t = cs[k / 2];
                const float y = v[k] * t.x - v[k + 1] * t.y;
                v[k + 1] = v[k] * t.y + v[k + 1] * t.x;
                v[k] = y;
            }
            store<TO, CH>(out + r.oo + c0, v, a.wide_out);
        }
    }
}

template <typename TI, typename TO, int CH>
cudaError_t launch(RotaryArgs a, bool in_place, cudaStream_t s) {
    constexpr int UPT = units_per_thread<TI>();
    auto rcp = [](int d) { return d > 1 ? (uint32_t)((1ull << 32) / d + 1) : 0u; };
    a.units[0] = a.half || CH == 1 ? a.rot_dim / 2 / CH : a.rot_dim / CH;
    a.units[1] = in_place ? 0 : (a.dim - a.rot_dim) / CH;
    a.heads_rcp = rcp(a.heads);
    long long ctas = 0;
    int slices = 1;
    for (int k = 0; k < 2; ++k) {
        a.ctas[k] = 0;
        if (a.units[k] == 0) continue;
        const int by_units = kThreads * UPT / a.units[k], by_table = k == 0 ? kTable / (a.rot_dim / 2) : by_units;
        a.per_cta[k] = max(1, min(by_units, by_table));
        a.units_rcp[k] = rcp(a.units[k]);
        const long long n = (a.vectors + a.per_cta[k] - 1) / a.per_cta[k];
        ctas += n;
        if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
        a.ctas[k] = (unsigned)n;
        slices = max(slices, (a.units[k] + kThreads * UPT - 1) / (kThreads * UPT));
    }
    const size_t table = sizeof(float2) * ((a.heads - 2 + (long long)a.per_cta[0]) / a.heads + 1) * (a.rot_dim / 2);
    rotary_kernel<TI, TO, CH><<<dim3((unsigned)ctas, slices), dim3(kThreads), table, s>>>(a);
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
    auto wide = [&](const csa_vectors &v) {  // chunks of eight float32 on 32-byte boundaries
        return v.dtype == CSA_F32 && reinterpret_cast<uintptr_t>(v.data) % 32 == 0 && (rows == 1 || v.row_stride % 8 == 0) &&
               (heads == 1 || v.head_stride % 8 == 0);
    };
    a.wide_x = wide(x);
    a.wide_out = wide(out);
    const bool vec = dim % 8 == 0 && rope.rot_begin % 8 == 0 && rope.rot_dim % (a.half ? 16 : 8) == 0 && aligned(x) &&
                     aligned(out);
    if (x.dtype == CSA_BF16)
        return out.dtype == CSA_BF16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(a, vec, in_place, s)
                                     : launch_types<__nv_bfloat16, float>(a, vec, in_place, s);
    return out.dtype == CSA_BF16 ? launch_types<float, __nv_bfloat16>(a, vec, in_place, s)
                                 : launch_types<float, float>(a, vec, in_place, s);
}

}  // namespace csa

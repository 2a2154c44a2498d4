// kda_rotary.hip - rotary position encoding of q and k on gfx950.
//
// Pure bandwidth: every element is read and written once.  A thread owns a group
// of channel pairs of one token, forms their angles once (64-bit product, reduced
// to a turn, then cos and sin in 32 bits) and walks the heads with them.
// 4 x 4096 tokens of 16 + 4 heads of 128 channels, half turned, bf16 (168 MB): 34 us,
// 4.9 TB/s; 40 us without the non-temporal stores.  With the angles in LDS and tokens,
// heads and granules walked in memory order it was 36 us.
#include "kda_attn_device.h"

namespace kda {

namespace {

constexpr double kInv2Pi = 0.15915494309189533577;

// cos and sin of position * frequency: the product in turns keeps 53 bits, and
// only its fraction is rounded to fp32 (the angle is off by at most pi 2^-24), as is the
// product of each with `scale`; sine and cosine in 64 bits are left out for their cost.
__device__ __forceinline__ void turn(double pos, double freq, float scale, float sign, float& a, float& b) {
    double x = pos * (freq * kInv2Pi);
    x -= rint(x);
    float s, c;
    sincospif((float)(2.0 * x), &s, &c);
    a = c * scale;
    b = s * scale * sign;
}

// Head h of a token: q's heads, then k's.
template <typename T>
__device__ __forceinline__ void head_ptrs(const RotaryArgs& a, size_t tok, int h, const T*& in, T*& out) {
    if (h < a.H) {
        in = reinterpret_cast<const T*>(a.q) + tok * a.ldq + (size_t)h * a.D;
        out = reinterpret_cast<T*>(a.q_out) + tok * a.ldqo + (size_t)h * a.D;
    } else {
        in = reinterpret_cast<const T*>(a.k) + tok * a.ldk + (size_t)(h - a.H) * a.D;
        out = reinterpret_cast<T*>(a.k_out) + tok * a.ldko + (size_t)(h - a.H) * a.D;
    }
}

__device__ __forceinline__ void store_once(void* p, const uint4& x) {
    __builtin_nontemporal_store(u32x4{x.x, x.y, x.z, x.w}, reinterpret_cast<u32x4*>(p));
}

}  // namespace

// Two 16-byte granules per thread and head: N pairs (or 2 N copied channels).
template <typename T>
__global__ __launch_bounds__(256) void kda_rotary_kernel(const RotaryArgs a, int units, int heads_per) {
    constexpr int N = Gran16<T>::N;
    const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
    const size_t tok = at / units;
    const int u = (int)(at % units);
    if (tok >= a.tokens) return;
    const int nrot = a.rot / (2 * N);       // units that turn; the others copy
    const bool turns = u < nrot;
    float ca[N], sa[N];
    int c0, c1;                              // first channels of the two granules
    if (turns) {
        const double pos = a.positions ? (double)a.positions[tok] : (double)(tok % a.T);
        const float sign = a.inverse ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < N; ++i) turn(pos, a.inv_freq[u * N + i], a.scale, sign, ca[i], sa[i]);
        c0 = a.interleaved ? 2 * N * u : N * u;
        c1 = a.interleaved ? c0 + N : c0 + a.rot / 2;
    } else {
        c0 = 2 * N * u;
        c1 = c0 + N;
    }
    const int h0 = blockIdx.y * heads_per, h1 = min(h0 + heads_per, a.H + a.HK);
    for (int h = h0; h < h1; ++h) {
        const T* in;
        T* out;
        head_ptrs(a, tok, h, in, out);
        const uint4 x = *reinterpret_cast<const uint4*>(in + c0), y = *reinterpret_cast<const uint4*>(in + c1);
        if (!turns) {
            if (in != out) {
                store_once(out + c0, x);
                store_once(out + c1, y);
            }
            continue;
        }
        float p[N], q[N];
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float x0 = Gran16<T>::get(x, 2 * i), x1 = Gran16<T>::get(x, 2 * i + 1);
                const float y0 = Gran16<T>::get(y, 2 * i), y1 = Gran16<T>::get(y, 2 * i + 1);
                p[2 * i] = ca[i] * x0 - sa[i] * x1;
                p[2 * i + 1] = sa[i] * x0 + ca[i] * x1;
                q[2 * i] = ca[N / 2 + i] * y0 - sa[N / 2 + i] * y1;
                q[2 * i + 1] = sa[N / 2 + i] * y0 + ca[N / 2 + i] * y1;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x0 = Gran16<T>::get(x, i), x1 = Gran16<T>::get(y, i);
                p[i] = ca[i] * x0 - sa[i] * x1;
                q[i] = sa[i] * x0 + ca[i] * x1;
            }
        }
        store_once(out + c0, Gran16<T>::pack(p));
        store_once(out + c1, Gran16<T>::pack(q));
    }
}

// Any even rot: one pair, or one copied channel, per thread and head.
template <typename T>
__global__ __launch_bounds__(256) void kda_rotary_pairs_kernel(const RotaryArgs a, int units, int heads_per) {
    const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
    const size_t tok = at / units;
    const int u = (int)(at % units);
    if (tok >= a.tokens) return;
    const bool turns = u < a.rot / 2;
    float ca = 1.f, sa = 0.f;
    int c0 = a.rot / 2 + u, c1 = c0;
    if (turns) {
        const double pos = a.positions ? (double)a.positions[tok] : (double)(tok % a.T);
        turn(pos, a.inv_freq[u], a.scale, a.inverse ? -1.f : 1.f, ca, sa);
        c0 = a.interleaved ? 2 * u : u;
        c1 = a.interleaved ? c0 + 1 : c0 + a.rot / 2;
    }
    const int h0 = blockIdx.y * heads_per, h1 = min(h0 + heads_per, a.H + a.HK);
    for (int h = h0; h < h1; ++h) {
        const T* in;
        T* out;
        head_ptrs(a, tok, h, in, out);
        if (!turns) {
            if (in != out) out[c0] = in[c0];
            continue;
        }
        const float x = to_f<T>(in[c0]), y = to_f<T>(in[c1]);
        out[c0] = from_f<T>(ca * x - sa * y);
        out[c1] = from_f<T>(sa * x + ca * y);
    }
}

template <typename T>
static hipError_t launch_rotary_t(const RotaryArgs& a, hipStream_t s) {
    constexpr int N = Gran16<T>::N;
    const bool wide = a.rot % (2 * N) == 0;  // both granules of every pair group are 16-byte aligned
    const int units = wide ? a.D / (2 * N) : a.rot / 2 + (a.D - a.rot);
    const int heads = a.H + a.HK;
    const size_t blocks = (a.tokens * units + 255) / 256;
    // few tokens: the heads are dealt over workgroups until the card is full
    size_t parts = blocks >= 1024 ? 1 : (1024 + blocks - 1) / blocks;
    if (parts > (size_t)heads) parts = heads;
    const int per = (heads + (int)parts - 1) / (int)parts;
    const dim3 grid((unsigned)blocks, (unsigned)((heads + per - 1) / per));
    if (wide) hipLaunchKernelGGL((kda_rotary_kernel<T>), grid, dim3(256), 0, s, a, units, per);
    else hipLaunchKernelGGL((kda_rotary_pairs_kernel<T>), grid, dim3(256), 0, s, a, units, per);
    return hipGetLastError();
}

hipError_t launch_rotary(int dt, const RotaryArgs& a, hipStream_t s) {
    return dt == 1 ? launch_rotary_t<bf16_t>(a, s) : launch_rotary_t<float>(a, s);
}

}  // namespace kda

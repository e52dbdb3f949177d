// attn_rotary.cu -- rotary positions: pair i of a row's first `width` channels
// is turned by the angle p * theta_i of its token's position p, in the "half"
// layout (pairs i, i + width / 2) or the interleaved one (pairs 2i, 2i + 1):
//     (x, y) -> amplitude * (x cos a - y sin a, x sin a + y cos a)
// and, for the gradient (transpose), by -a.  Channels behind `width` are
// copied.
//
// Angles.  theta_i arrives as a 64-bit fixed-point fraction of a turn per
// position, so that the product with an integer position wraps at whole turns
// by itself: the angle is exact to 2^-64 of a turn times the position, at any
// 32-bit position, without a table of positions and without fp64.  Its upper
// 32 bits are reduced to an eighth of a turn around the nearest quarter, where
// sincospif has less than one unit in the last place to lose.
//
// What bounds it: the bytes of the rows.  A CTA takes a few whole tokens:
// it computes their sines and cosines once into shared memory (for all heads
// of q and k together), while the first rows are already on their way, and
// then streams the rows with 16-byte loads and stores, two items (of two
// vectors each) in flight per thread and four CTAs an SM.  8192 tokens of 40
// heads of 128 in bf16, 168 MB, take 30 us: 5.5 TB/s, 82 % of the measured copy
// rate; one token of 32 sequences takes 2.6 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "attn_internal.h"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;  // tokens of a CTA at most
constexpr int kCtasPerSm = 4;
constexpr int kUnroll = 2;      // items a thread has in flight

struct RotaryParams {
    attn_heads q, k;        // k.H = 0: q alone
    const uint64_t *turns;  // [width / 2] fractions of a turn per position
    const int32_t *pos;
    int pos_tokens;  // 1: pos [B][S]; 0: pos [B], the first token's
    int64_t tokens;  // B * S
    int S, d, width, cpr;  // cpr: items of a row
    int T;                 // tokens of a CTA
    int HB, n_hb;          // heads of a CTA (q and k together), head blocks
    float amplitude;
    int transpose;
    int *status;
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// A vector as fp32 values and back, 16-bit ones in pairs.
template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V> &x, float *f) {
    if constexpr (V == 1 || sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f(x.e[i]);
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(x.e);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const uint32_t u = w[i];
            float2 p;
            if constexpr (std::is_same<T, __half>::value)
                p = __half22float2(*reinterpret_cast<const __half2 *>(&u));
            else
                p = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ void pack(const float *f, Vec<T, V> &x) {
    if constexpr (V == 1 || sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) x.e[i] = from_f<T>(f[i]);
    } else {
        uint32_t *w = reinterpret_cast<uint32_t *>(x.e);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
}

// cos and sin of pair i of a token, in the order the items read them: the
// VEC pairs of item c in groups of four, group g of all items side by side
// (consecutive items then read consecutive 16-byte words).
template <int V>
__device__ __forceinline__ int place(int i, int items) {
    constexpr int W = V < 4 ? V : 4;
    const int c = i / V, e = i % V;
    return ((e / W) * items + c) * W + e % W;
}

template <typename T, int V, bool kHalf>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
attn_rotary_kernel(const RotaryParams p) {
    extern __shared__ __align__(16) float table[];  // [T][2][width / 2]: cosines, sines
    __shared__ int64_t base[kMaxTokens][4];         // offsets of a token's rows: q in, q out, k in, k out
    const int half = p.width / 2, turned = half / V;  // items of a row that are turned
    const int64_t n0 = (int64_t)blockIdx.x * p.T;
    const int nt = (int)min((int64_t)p.T, p.tokens - n0);
    const int h0 = blockIdx.y * p.HB, nh = min(p.HB, p.q.H + p.k.H - h0);
    const int total = nt * nh * p.cpr;

    if (threadIdx.x < nt) {
        const int64_t n = n0 + threadIdx.x;
        const int64_t b = n / p.S, s = n - b * p.S;
        base[threadIdx.x][0] = b * p.q.in_stride[0] + s * p.q.in_stride[2];
        base[threadIdx.x][1] = b * p.q.out_stride[0] + s * p.q.out_stride[2];
        base[threadIdx.x][2] = b * p.k.in_stride[0] + s * p.k.in_stride[2];
        base[threadIdx.x][3] = b * p.k.out_stride[0] + s * p.k.out_stride[2];
    }
    __syncthreads();

    // This thread's items: (token, head, item of the row), items fastest, and the
    // step of kThreads items in the same digits, so that none is divided for again.
    int c = threadIdx.x % p.cpr, h, t;
    {
        const int r = threadIdx.x / p.cpr;
        h = r % nh;
        t = r / nh;
    }
    const int dc = kThreads % p.cpr, dh = (kThreads / p.cpr) % nh, dt = kThreads / p.cpr / nh;
    int it = threadIdx.x;

    struct Item {
        Vec<T, V> a, b;
        T *out;  // where a goes; b goes `apart` of its item behind it
        int c, t;
    };
    auto apart = [&](int c) { return kHalf && c < turned ? half : V; };
    auto load = [&](Item &x) {
        const int head = h0 + h;
        const bool is_k = head >= p.q.H;
        const attn_heads &w = is_k ? p.k : p.q;
        const int hh = is_k ? head - p.q.H : head;
        const T *in = (const T *)w.in + base[t][is_k ? 2 : 0] + hh * w.in_stride[1];
        T *out = (T *)w.out + base[t][is_k ? 3 : 1] + hh * w.out_stride[1];
        // channels of the two vectors
        const int ca = c >= turned ? p.width + (c - turned) * 2 * V : kHalf ? c * V : c * 2 * V;
        const int cb = ca + apart(c);
        x.c = c;
        x.t = t;
        x.out = out + ca;
        if (in_bounds(hh < w.H && cb + V <= p.d && n0 + t < p.tokens, p.status)) {
            x.a = *reinterpret_cast<const Vec<T, V> *>(in + ca);
            x.b = *reinterpret_cast<const Vec<T, V> *>(in + cb);
        }
        c += dc;
        h += dh;
        t += dt;
        if (c >= p.cpr) { c -= p.cpr; ++h; }
        if (h >= nh) { h -= nh; ++t; }
    };
    auto finish = [&](Item &x) {
        if (x.c < turned) {
            const float *cs = table + (size_t)x.t * p.width, *sn = cs + half;
            float f[2 * V];  // both vectors
            unpack(x.a, f);
            unpack(x.b, f + V);
            constexpr int W = V < 4 ? V : 4;
#pragma unroll
            for (int g = 0; g < V / W; ++g) {
                const int at = (g * turned + x.c) * W;
                const Vec<float, W> cv = *reinterpret_cast<const Vec<float, W> *>(cs + at);
                const Vec<float, W> sv = *reinterpret_cast<const Vec<float, W> *>(sn + at);
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    // pair g W + e: the same place of both vectors, or neighbours
                    const int i = g * W + e, a = kHalf ? i : 2 * i, b = kHalf ? V + i : 2 * i + 1;
                    const float u = f[a], v = f[b];
                    f[a] = u * cv.e[e] - v * sv.e[e];
                    f[b] = u * sv.e[e] + v * cv.e[e];
                }
            }
            pack(f, x.a);
            pack(f + V, x.b);
        }
        if (in_bounds(x.c < p.cpr && x.t < nt, p.status)) {
            *reinterpret_cast<Vec<T, V> *>(x.out) = x.a;
            *reinterpret_cast<Vec<T, V> *>(x.out + apart(x.c)) = x.b;
        }
    };

    // the first rows are on their way while the angles are computed
    Item x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (it + u * kThreads < total) load(x[u]);

    for (int j = threadIdx.x; j < nt * half; j += kThreads) {
        const int tt = j / half, i = j - tt * half;
        const int64_t g = n0 + tt, b = g / p.S;
        // wraps modulo 2^32, as positions do
        const uint32_t at = p.pos_tokens ? (uint32_t)p.pos[g] : (uint32_t)p.pos[b] + (uint32_t)(g - b * p.S);
        const uint64_t turn = (uint64_t)(int64_t)(int32_t)at * p.turns[i] + 0x80000000ull;
        const uint32_t hi = (uint32_t)(turn >> 32);
        const uint32_t quarter = (hi + 0x20000000u) >> 30;
        const float r = (float)(int32_t)(hi - (quarter << 30)) * 0x1p-31f;  // half turns, |r| <= 1/4
        float s0, c0;
        sincospif(r, &s0, &c0);
        const float cc = quarter & 1 ? s0 : c0, ss = quarter & 1 ? c0 : s0;
        const float co = (quarter == 1 || quarter == 2) ? -cc : cc;
        const float si = quarter >= 2 ? -ss : ss;
        float *row = table + (size_t)tt * p.width;
        const int w = place<V>(i, turned);
        row[w] = co * p.amplitude;
        row[half + w] = (p.transpose ? -si : si) * p.amplitude;
    }
    __syncthreads();

    // each item finished makes room for the next one's loads
    while (it < total) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (it + u * kThreads < total) finish(x[u]);
            if (it + (u + kUnroll) * kThreads < total) load(x[u]);
        }
        it += kUnroll * kThreads;
    }
}

template <typename T, int V, bool kHalf>
int launch_v(RotaryParams p, cudaStream_t stream) {
    p.cpr = p.d / (2 * V);
    const int sms = device_sm_count();
    if (sms <= 0) return ATTN_ERR_CUDA;
    const int H = p.q.H + p.k.H;
    // Tokens of a CTA: whole rounds of resident CTAs with equal shares of up to 32
    // tokens, so that a thread has a long row of items whose loads and stores overlap
    // and no round is left for a few CTAs (8192 tokens of 40 heads, three CTAs an SM:
    // 512 CTAs of 16 tokens took 64 us, 456 of 18 took 46); a single token of many
    // heads is cut by heads while SMs are free.
    const int64_t items = (int64_t)H * p.cpr;
    const int64_t places = (int64_t)kCtasPerSm * sms;
    int64_t most = 8192 / p.width;  // 32 KB of angles
    if (most > kMaxTokens) most = kMaxTokens;
    const int64_t rounds = (p.tokens + places * most - 1) / (places * most);
    p.T = (int)((p.tokens + places * rounds - 1) / (places * rounds));
    const int64_t gx = (p.tokens + p.T - 1) / p.T;
    int64_t cuts = 1;
    if (gx < sms) {
        cuts = sms / gx;
        const int64_t whole = (items + kThreads - 1) / kThreads;  // CTAs that leave each thread an item
        if (cuts > whole) cuts = whole;
    } else {
        // many heads: no CTA walks more than 32 rounds
        cuts = (items * p.T + kThreads * 32 - 1) / (kThreads * 32);
    }
    if (cuts > H) cuts = H;
    if (cuts > 65535) cuts = 65535;
    p.HB = (int)((H + cuts - 1) / cuts);
    p.n_hb = (H + p.HB - 1) / p.HB;
    if (gx > INT32_MAX) return ATTN_ERR_INVALID_ARG;
    const size_t smem = (size_t)p.T * p.width * sizeof(float);
    p.status = status_word_device_ptr();
    if (!p.status) return ATTN_ERR_CUDA;
    attn_rotary_kernel<T, V, kHalf><<<dim3((unsigned)gx, (unsigned)p.n_hb), kThreads, smem, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

template <typename T, int V>
int launch_layout(const RotaryParams &p, bool interleaved, cudaStream_t stream) {
    return interleaved ? launch_v<T, V, false>(p, stream) : launch_v<T, V, true>(p, stream);
}

// Widest vectors that both halves of a pair's item and the copied channels allow:
// V elements where 2 V divides the turned and all channels and V every stride and address.
template <typename T>
int launch_type(const RotaryParams &p, bool interleaved, cudaStream_t stream) {
    auto fits = [&](int V) {
        if (p.width % (2 * V) != 0 || p.d % (2 * V) != 0) return false;
        for (const attn_heads *w : {&p.q, &p.k}) {
            if (w->H == 0) continue;
            if ((uintptr_t)w->in % (V * sizeof(T)) != 0 || (uintptr_t)w->out % (V * sizeof(T)) != 0)
                return false;
            for (int i = 0; i < 3; ++i)
                if (w->in_stride[i] % V != 0 || w->out_stride[i] % V != 0) return false;
        }
        return true;
    };
    if constexpr (sizeof(T) == 2) {
        if (fits(8)) return launch_layout<T, 8>(p, interleaved, stream);
    }
    if (fits(4)) return launch_layout<T, 4>(p, interleaved, stream);
    return launch_layout<T, 1>(p, interleaved, stream);
}

}  // namespace

int launch_rotary(const attn_heads &q, const attn_heads *k, const uint64_t *turns, int width,
                  bool interleaved, float amplitude, bool transpose, const int32_t *pos,
                  int pos_tokens, int B, int S, int d, int dtype, cudaStream_t stream) {
    RotaryParams p{};
    p.q = q;
    if (k) p.k = *k;
    else p.k.H = 0;
    p.turns = turns;
    p.pos = pos;
    p.pos_tokens = pos_tokens;
    p.tokens = (int64_t)B * S;
    p.S = S;
    p.d = d;
    p.width = width;
    p.amplitude = amplitude;
    p.transpose = transpose;
    if (dtype == 0) return launch_type<float>(p, interleaved, stream);
    if (dtype == 1) return launch_type<__nv_bfloat16>(p, interleaved, stream);
    return launch_type<__half>(p, interleaved, stream);
}

}  // namespace attn

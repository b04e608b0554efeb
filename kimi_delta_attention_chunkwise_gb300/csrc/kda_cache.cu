// kda_cache.cu -- new tokens' keys and values into the paged cache, with
// queries and keys rotated by their positions on the way.
//
// Pair (a, b) of a row's channels turns by the angle its position and pair
// index give:  y_a = x_a cos - x_b sin,  y_b = x_b cos + x_a sin.  The two
// products and the sum of each are rounded separately (no fused multiply-add),
// so a result is the same wherever its pair sits; bf16 results are rounded
// once more, at the end.
//
// Memory-bound: every input byte is read once and every output byte written
// once, in 16-byte vectors.  A work unit is two vectors of one head's row:
// the two whose channels pair up (halves), or any two neighbours
// (interleaved pairs, and channels past rot_dim).  A CTA takes TOK tokens:
// one thread per token looks its position and page up (two dependent reads)
// while the others' first vectors are already on their way, then all threads
// walk the CTA's units (heads of q, then k, then v), one unit ahead.
//
// A cache of 8-bit codes (kda_cache_append_q8) holds a row of a head as
//     code = rint(x * (127 / top)),   scale = top / 127,   top = max |x|
// of the rotated fp32 row, with each of these operations rounded to fp32: what
// the codes stand for is off by half a scale at most (and fp32's rounding).
// top is the maximum over the row's neighbouring lanes, as integers, in which
// infinities and NaN are above every number.  A CTA takes one token; a thread has
// the same unit of every so-many-th row, so that it loads its angles once, and two
// rows' vectors at a time.  More CTAs to an SM count for more than more rows in
// flight (16384 tokens, 32/8 heads, d = 128, the values that the codes stand for
// among the outputs: 8 CTAs 76.5 us, 5.8 TB/s; 7 with three rows 77.5, 6 79.4; one
// row and 8 78.8; 9 spill, 84).
#include <cstdint>
#include <cuda_bf16.h>

#include "kda_attn.cuh"

namespace kda {
namespace {

// Up to so many tokens a CTA of 256 threads takes one (256 tokens, 32/8 heads:
// 3.2 us); beyond, CTAs of 128 threads take two (16384 tokens: 73 us, 6.1 TB/s,
// where a plain copy of as many bytes runs at 5.3; 4 tokens to 256 threads:
// 78 us).
constexpr int kFewTokens = 1024;

template <typename T>
struct Row;  // 16 bytes of a row as floats
template <>
struct Row<float> {
    static constexpr int V = 4;
    __device__ static void unpack(const uint4 &x, float (&f)[4]) {
        f[0] = __uint_as_float(x.x); f[1] = __uint_as_float(x.y);
        f[2] = __uint_as_float(x.z); f[3] = __uint_as_float(x.w);
    }
    __device__ static uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};
template <>
struct Row<__nv_bfloat16> {
    static constexpr int V = 8;
    __device__ static void unpack(const uint4 &x, float (&f)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ static uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float ya = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    const float yb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = ya;
    b = yb;
}

// The sequence that holds token t: the last s with cu[s] <= t (cu
// non-decreasing; empty sequences hold nothing).
__device__ __forceinline__ int32_t seq_of_token(const int32_t *cu, int32_t N, int32_t t) {
    int32_t lo = 0, hi = N - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One token's place, looked up once per CTA.
struct Place {
    int32_t pos;      // < 0: the token is skipped whole
    int64_t page;     // row offset (in rows of one head) of the cache slot, < 0: not cached
};

__device__ Place find_place(const AppendArgs &a, int32_t t) {
    Place p;
    p.pos = -1;
    p.page = -1;
    if (t >= a.T) return p;
    int32_t s = 0, first = 0;
    if (a.one_each) {
        s = t;
        first = t;
    } else if (a.cu_seqlens) {
        s = seq_of_token(a.cu_seqlens, a.N, t);
        first = a.cu_seqlens[s];
        if (t < first || t >= a.cu_seqlens[s + 1]) return p;  // outside every sequence
        first = max(first, 0);
    }
    const int64_t pos = (int64_t)a.cache_lens[s] + (t - first);
    const int32_t size = 1 << a.page_shift;
    if (pos < 0 || (pos >> a.page_shift) >= a.max_pages || (a.rope && pos >= a.positions)) {
        *a.status = KDA_ERR_INVALID_ARG;
        return p;
    }
    const int32_t page = a.block_table[(int64_t)s * a.max_pages + (pos >> a.page_shift)];
    if (page >= a.num_pages) {
        *a.status = KDA_ERR_INVALID_ARG;
        return p;
    }
    p.pos = (int32_t)pos;
    if (page >= 0) p.page = (int64_t)page * a.HKV * size + (pos & (size - 1));
    return p;
}

// A unit: two 16-byte vectors of one head's row.
struct Unit {
    int32_t tk, head, c0, c1;  // token of the CTA, row (q, k, v heads), first channels
    bool halves;               // the two vectors pair up
};

template <typename T, int D, int TOK, int kThreads>
__global__ void __launch_bounds__(kThreads, TOK == 1 ? 1 : 9) cache_append_kernel(const AppendArgs a) {
    constexpr int V = Row<T>::V;
    constexpr int UNITS = D / V / 2;  // units per head row
    __shared__ Place place[TOK];
    const int32_t t0 = blockIdx.x * TOK;
    const int32_t rows = a.HQ + 2 * a.HKV;
    const int32_t half = a.rot >> 1;
    const int32_t total = min(TOK, a.T - t0) * rows * UNITS;
    auto unit_of = [&](int32_t i) {
        Unit w;
        const int32_t u = i % UNITS, r = i / UNITS;
        w.tk = r / rows;
        w.head = r - w.tk * rows;
        w.halves = a.rot > 0 && !a.interleaved && u * V < half;
        w.c0 = w.halves ? u * V : 2 * u * V;
        w.c1 = w.halves ? w.c0 + half : w.c0 + V;
        return w;
    };
    // inputs do not wait for the look-up: every row of [0, T) may be read
    auto load = [&](int32_t i, uint4 &x0, uint4 &x1) {
        const Unit w = unit_of(i);
        const int64_t t = t0 + w.tk;
        const T *src;
        if (w.head < a.HQ) {
            src = static_cast<const T *>(a.q) + t * a.q_stride + (int64_t)w.head * D;
        } else if (w.head < a.HQ + a.HKV) {
            src = static_cast<const T *>(a.k) + t * a.k_stride + (int64_t)(w.head - a.HQ) * D;
        } else {
            src = static_cast<const T *>(a.v) + t * a.v_stride + (int64_t)(w.head - a.HQ - a.HKV) * D;
        }
        x0 = *reinterpret_cast<const uint4 *>(src + w.c0);
        x1 = *reinterpret_cast<const uint4 *>(src + w.c1);
    };
    auto finish = [&](int32_t i, uint4 x0, uint4 x1) {
        const Unit w = unit_of(i);
        const Place p = place[w.tk];
        if (p.pos < 0) return;
        const int64_t t = t0 + w.tk;
        T *dst0 = nullptr, *dst1 = nullptr;  // contiguous output, cache row
        bool rotate = w.c0 < a.rot;
        if (w.head < a.HQ) {
            dst0 = static_cast<T *>(a.q_out) + (t * a.HQ + w.head) * D;
        } else {
            const int32_t h = w.head - a.HQ;
            const bool is_k = h < a.HKV;
            const int32_t kh = is_k ? h : h - a.HKV;
            const int64_t row = (p.page + ((int64_t)kh << a.page_shift)) * D;
            if (p.page >= 0) dst1 = static_cast<T *>(is_k ? a.k_cache : a.v_cache) + row;
            if (is_k && a.k_out) dst0 = static_cast<T *>(a.k_out) + (t * a.HKV + kh) * D;
            rotate = rotate && is_k;
        }
        if (rotate) {
            const float *cs = a.rope + (int64_t)p.pos * a.rot;
            float f0[V], f1[V], c[V], s[V];
            Row<T>::unpack(x0, f0);
            Row<T>::unpack(x1, f1);
            // the angles of the unit's V pairs: halves: pairs c0 .. c0 + V - 1;
            // interleaved: c0 / 2 .. (both vectors lie inside rot_dim, a
            // multiple of 2 V)
            const float *ca = cs + (w.halves ? w.c0 : w.c0 / 2), *sa = ca + half;
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 cv = __ldg(reinterpret_cast<const float4 *>(ca + j));
                const float4 sv = __ldg(reinterpret_cast<const float4 *>(sa + j));
                c[j] = cv.x; c[j + 1] = cv.y; c[j + 2] = cv.z; c[j + 3] = cv.w;
                s[j] = sv.x; s[j + 1] = sv.y; s[j + 2] = sv.z; s[j + 3] = sv.w;
            }
            if (w.halves) {
#pragma unroll
                for (int j = 0; j < V; ++j) turn(f0[j], f1[j], c[j], s[j]);
            } else {
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    turn(f0[2 * j], f0[2 * j + 1], c[j], s[j]);
                    turn(f1[2 * j], f1[2 * j + 1], c[V / 2 + j], s[V / 2 + j]);
                }
            }
            x0 = Row<T>::pack(f0);
            x1 = Row<T>::pack(f1);
        }
        if (dst0) {
            *reinterpret_cast<uint4 *>(dst0 + w.c0) = x0;
            *reinterpret_cast<uint4 *>(dst0 + w.c1) = x1;
        }
        if (dst1) {
            *reinterpret_cast<uint4 *>(dst1 + w.c0) = x0;
            *reinterpret_cast<uint4 *>(dst1 + w.c1) = x1;
        }
    };
    // the next unit's vectors are on their way while this one's are worked on
    uint4 x0 = {}, x1 = {}, y0 = {}, y1 = {};
    if ((int32_t)threadIdx.x < total) load(threadIdx.x, x0, x1);
    if (threadIdx.x < TOK) place[threadIdx.x] = find_place(a, t0 + threadIdx.x);
    __syncthreads();
    for (int32_t i = threadIdx.x; i < total; i += kThreads) {
        if (i + kThreads < total) load(i + kThreads, y0, y1);
        finish(i, x0, x1);
        x0 = y0;
        x1 = y1;
    }
}

// A row's codes and what they stand for.
constexpr float kSmallest = 0x1p-100f;  // (below it, 127 / top might not be a number)
struct Coder {
    float scale, turn;
    // `top`: the bits of the row's largest magnitude
    __device__ explicit Coder(uint32_t top) {
        const float t = __uint_as_float(top);
        scale = __fdiv_rn(t, 127.f);
        turn = __fdiv_rn(127.f, t);
        if (top >= 0x7F800000u) {  // an infinity or a NaN: no code stands for it
            scale = __uint_as_float(0x7FC00000u);
            turn = 0.f;
        } else if (t < kSmallest) {
            scale = turn = 0.f;
        }
    }
    // (x is finite where turn is not 0)
    __device__ float code(float x) const { return turn == 0.f ? 0.f : rintf(__fmul_rn(x, turn)); }
};
template <int V>
__device__ __forceinline__ void store_codes(int8_t *to, const float (&c)[V]) {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        // a whole number from -127 to 127 above 1.5 * 2^23 is the sum's low byte
        const float *x = c + 4 * i;
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(x[j] + 12582912.f);
        w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(to) = w[0];
}

// (8 CTAs to an SM: 64 registers, bf16 rows spill 8-28 bytes of them; 9 CTAs cost more)
template <typename T, int D, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 128 ? 8 : 1) cache_append_q8_kernel(const AppendArgs a) {
    constexpr int V = Row<T>::V;
    constexpr int UNITS = D / V / 2;        // units per head row
    constexpr int STEP = kThreads / UNITS;  // rows abreast
    constexpr int B = 2;                    // rows of a thread in flight
    __shared__ Place place;
    const int32_t t = blockIdx.x, half = a.rot >> 1;
    const int32_t rows = a.HQ + 2 * a.HKV;
    const int32_t u = (int32_t)threadIdx.x % UNITS, r0 = (int32_t)threadIdx.x / UNITS;
    // the thread's two vectors of a row: the two whose channels pair up, or neighbours
    const bool halves = a.rot > 0 && !a.interleaved && u * V < half;
    const int32_t c0 = halves ? u * V : 2 * u * V, c1 = halves ? c0 + half : c0 + V;
    const bool turns = c0 < a.rot;
    float cs[V], sn[V];  // the angles of the unit's pairs
    Place p;
    for (int32_t rb = 0; rb < rows; rb += STEP * B) {
        // inputs do not wait for the look-up: every row of [0, T) may be read
        uint4 x0[B], x1[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int32_t r = rb + r0 + b * STEP;
            if (r >= rows) continue;
            const T *src;
            if (r < a.HQ) src = static_cast<const T *>(a.q) + t * a.q_stride + (int64_t)r * D;
            else if (r < a.HQ + a.HKV)
                src = static_cast<const T *>(a.k) + t * a.k_stride + (int64_t)(r - a.HQ) * D;
            else
                src = static_cast<const T *>(a.v) + t * a.v_stride + (int64_t)(r - a.HQ - a.HKV) * D;
            x0[b] = *reinterpret_cast<const uint4 *>(src + c0);
            x1[b] = *reinterpret_cast<const uint4 *>(src + c1);
        }
        if (rb == 0) {
            if (threadIdx.x == 0) place = find_place(a, t);
            __syncthreads();
            p = place;
            if (p.pos < 0) return;
            if (turns) {
                const float *ca = a.rope + (int64_t)p.pos * a.rot + (halves ? c0 : c0 / 2);
#pragma unroll
                for (int j = 0; j < V; j += 4) {
                    const float4 c = __ldg(reinterpret_cast<const float4 *>(ca + j));
                    const float4 s = __ldg(reinterpret_cast<const float4 *>(ca + half + j));
                    cs[j] = c.x; cs[j + 1] = c.y; cs[j + 2] = c.z; cs[j + 3] = c.w;
                    sn[j] = s.x; sn[j + 1] = s.y; sn[j + 2] = s.z; sn[j + 3] = s.w;
                }
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int32_t r = rb + r0 + b * STEP;
            const bool here = r < rows, is_q = r < a.HQ, is_k = !is_q && r < a.HQ + a.HKV;
            if (!__any_sync(0xffffffffu, here)) break;
            float f0[V], f1[V];
            Row<T>::unpack(x0[b], f0);
            Row<T>::unpack(x1[b], f1);
            const bool turned = turns && (is_q || is_k);
            if (turned) {
                if (halves) {
#pragma unroll
                    for (int j = 0; j < V; ++j) turn(f0[j], f1[j], cs[j], sn[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) {
                        turn(f0[2 * j], f0[2 * j + 1], cs[j], sn[j]);
                        turn(f1[2 * j], f1[2 * j + 1], cs[V / 2 + j], sn[V / 2 + j]);
                    }
                }
            }
            // the row as it is turned (what is not is copied: packing it again would
            // change a NaN's bits)
            auto put_turned = [&](T *row) {
                *reinterpret_cast<uint4 *>(row + c0) = turned ? Row<T>::pack(f0) : x0[b];
                *reinterpret_cast<uint4 *>(row + c1) = turned ? Row<T>::pack(f1) : x1[b];
            };
            if (here && is_q) put_turned(static_cast<T *>(a.q_out) + ((int64_t)t * a.HQ + r) * D);
            // (most warps have queries alone)
            if (!__any_sync(0xffffffffu, here && !is_q)) continue;
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                top = max(top, max(__float_as_uint(f0[j]) & 0x7FFFFFFFu,
                                   __float_as_uint(f1[j]) & 0x7FFFFFFFu));
#pragma unroll
            for (int o = 1; o < UNITS; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (here && !is_q) {
                const int32_t kh = r - a.HQ - (is_k ? 0 : a.HKV);
                const int64_t out = ((int64_t)t * a.HKV + kh) * D;
                if (is_k && a.k_out) put_turned(static_cast<T *>(a.k_out) + out);
                const Coder coder(top);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    f0[j] = coder.code(f0[j]);
                    f1[j] = coder.code(f1[j]);
                }
                if (p.page >= 0) {
                    const int64_t row = p.page + ((int64_t)kh << a.page_shift);
                    int8_t *to = static_cast<int8_t *>(is_k ? a.k_cache : a.v_cache) + row * D;
                    store_codes<V>(to + c0, f0);
                    store_codes<V>(to + c1, f1);
                    if (u == 0) (is_k ? a.k_scale : a.v_scale)[row] = coder.scale;
                }
                T *stored = static_cast<T *>(is_k ? a.k_stored : a.v_stored);
                if (stored) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        f0[j] = __fmul_rn(f0[j], coder.scale);
                        f1[j] = __fmul_rn(f1[j], coder.scale);
                    }
                    *reinterpret_cast<uint4 *>(stored + out + c0) = Row<T>::pack(f0);
                    *reinterpret_cast<uint4 *>(stored + out + c1) = Row<T>::pack(f1);
                }
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch_t(const AppendArgs &a, cudaStream_t stream) {
    if (a.T <= kFewTokens) {
        cache_append_kernel<T, D, 1, 256><<<(unsigned)a.T, 256, 0, stream>>>(a);
    } else {
        cache_append_kernel<T, D, 2, 128><<<(unsigned)(a.T / 2 + a.T % 2), 128, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(const AppendArgs &a, cudaStream_t stream) {
    switch (a.D) {
        case 16: return launch_t<T, 16>(a, stream);
        case 32: return launch_t<T, 32>(a, stream);
        case 64: return launch_t<T, 64>(a, stream);
        case 128: return launch_t<T, 128>(a, stream);
    }
    return cudaErrorInvalidValue;
}

template <typename T, int D>
cudaError_t launch_q8_t(const AppendArgs &a, cudaStream_t stream) {
    if (a.T <= kFewTokens) cache_append_q8_kernel<T, D, 256><<<(unsigned)a.T, 256, 0, stream>>>(a);
    else cache_append_q8_kernel<T, D, 128><<<(unsigned)a.T, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_q8_d(const AppendArgs &a, cudaStream_t stream) {
    switch (a.D) {
        case 16: return launch_q8_t<T, 16>(a, stream);
        case 32: return launch_q8_t<T, 32>(a, stream);
        case 64: return launch_q8_t<T, 64>(a, stream);
        case 128: return launch_q8_t<T, 128>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t stream) {
    if (a.dtype == KDA_DTYPE_BF16) return launch_d<__nv_bfloat16>(a, stream);
    return launch_d<float>(a, stream);
}

cudaError_t launch_cache_append_q8(const AppendArgs &a, cudaStream_t stream) {
    if (a.dtype == KDA_DTYPE_BF16) return launch_q8_d<__nv_bfloat16>(a, stream);
    return launch_q8_d<float>(a, stream);
}

}  // namespace kda

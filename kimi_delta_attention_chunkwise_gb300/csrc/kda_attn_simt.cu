// kda_attn_simt.cu -- causal attention over packed prompts in fp32 on CUDA
// cores: every supported shape, and the engine of fp32 inputs.
//
//     z_ij = scale <q_i, k_j>  (j <= i),   o_i = sum_j e^{z_ij} v_j / sum_j e^{z_ij}
//
// One pass over the keys with a running maximum and sum per row, in base 2
// (z scaled by log2 e).  The rows of a tile are (token, query head) pairs of
// one key-value head, token-major, so grouped heads share every key and value
// that is brought in and a group of any size fills its tiles.
//
// A group of threads owns ROWS rows and walks the keys in tiles of 64: a thread
// computes an MI x 4 block of scores (rows MI ty + a, keys tx + 16 b) and D / 16
// columns of MI output rows.  The 16 threads of a row share its statistics
// through shuffles; the weights pass through shared memory.  The keys of the
// next tile are brought in beside the softmax and the values' product, the
// values beside the scores.  GROUPS groups of a CTA share the rows, each taking
// every GROUPS-th key tile, and join their states at the end.
//
// What bounds it: shared memory's reads: per 4 channels a thread reads MI + 4
// vectors of 16 bytes for 8 MI two-wide multiply-adds, so blocks of 8 x 4 run
// faster than 4 x 4 where the GPU is full (4 x 1000 tokens, 8/2 heads, d = 64:
// 118 us, 4 x 4 169; one prompt of 4000 tokens, d = 128: 699 us, 47 TFLOP/s of
// fp32, 4 x 4 816).  Four sizes (launch_t):
//
//   64 rows, two groups, 8 x 4: where those tiles fill the GPU.
//   64 rows, one group, 4 x 4, two CTAs to an SM: the same, but with sequences
//     of one key tile on average, which leave a second group idle (100 x 30
//     tokens, 8/2 heads, d = 64: 17.5 us, two groups 28).
//   16 rows, two groups, 4 x 4, two CTAs to an SM: smaller problems, where the
//     longest tile's steps in a row decide (1025 tokens of 3 sequences, 6/2
//     heads, d = 64: 25 us, 32 rows and four groups 28, 64 rows 45-54).
//   32 rows, two groups, 4 x 4: the same for D = 128, as far as shared memory
//     goes (those 1025 tokens: 47 us, 16 rows 49-70, 64 rows 76-92).
#include <cstdint>
#include <cuda_bf16.h>
#include <type_traits>

#include "kda_attn_common.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kKeys = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D>
constexpr int kq_stride() { return D + 4; }  // rows 4 banks apart: 16-byte reads without conflicts
constexpr int kPStride = kKeys + 4;

// Whether the weights have a place of their own in a group's tiles (else they
// overwrite the keys, whose next tile then cannot come early): two CTAs with 64
// rows of D = 128 leave them none.  Floats of a group's keys and weights, and
// bytes of a CTA.
template <int D, int ROWS, int GROUPS>
constexpr bool weights_apart() { return !(D == 128 && ROWS == 64 && GROUPS == 1); }
template <int D, int ROWS, int GROUPS>
constexpr int key_floats() {
    return kKeys * kq_stride<D>() + (weights_apart<D, ROWS, GROUPS>() ? ROWS * kPStride : 0);
}
template <int D, int ROWS, int GROUPS>
constexpr size_t smem_bytes() {
    return (ROWS * kq_stride<D>() + GROUPS * (key_floats<D, ROWS, GROUPS>() + kKeys * D)) * sizeof(float);
}

// 4 elements of a row to shared memory as floats (zeros without `in`): fp32
// asynchronously, in the thread's next group of copies
__device__ __forceinline__ void bring4(float *to, const float *from, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u),
                       __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xFFFF0000u));
}
__device__ __forceinline__ void bring4(float *to, const __nv_bfloat16 *from, bool in) {
    *reinterpret_cast<float4 *>(to) = in ? load4(from) : make_float4(0.f, 0.f, 0.f, 0.f);
}

template <typename T, int D, int ROWS, int GROUPS, int MI, int OCC>
__global__ void __launch_bounds__(GROUPS * ROWS / MI * 16, OCC)
attn_simt_kernel(const AttnArgs a) {
    constexpr int kRows = ROWS, kGroup = ROWS / MI * 16, kThreads = GROUPS * kGroup;
    constexpr int KS = kq_stride<D>();
    constexpr bool kApart = weights_apart<D, ROWS, GROUPS>();
    constexpr int CW = D >= 64 ? 4 : D / 16;      // columns of one vector
    constexpr int CN = D >= 64 ? D / 64 : 1;      // vectors per thread, 64 columns apart
    extern __shared__ float smem[];
    const int group = threadIdx.x / kGroup, tid = threadIdx.x % kGroup, tx = tid & 15, ty = tid >> 4;
    float *sq = smem;
    float *sk = smem + kRows * KS + group * (key_floats<D, ROWS, GROUPS>() + kKeys * D);
    float *sp = sk + (kApart ? kKeys * KS : 0);
    float *sv = sk + key_floats<D, ROWS, GROUPS>();
    __shared__ SeqTile s_tile;
    __shared__ int s_found;
    auto sync_group = [&]() {
        if (GROUPS == 1) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kGroup) : "memory");
    };
    if (threadIdx.x < 32) {
        SeqTile t;
        TileCursor cursor;
        const bool ok = find_seq_tile(a.cu_seqlens, a.N, a.T, (uint32_t)a.G, (uint32_t)kRows,
                                      blockIdx.x / a.HKV, cursor, t);
        if (threadIdx.x == 0) {
            s_found = ok;
            if (ok) s_tile = t;
        }
    }
    __syncthreads();
    if (!s_found) return;
    const SeqTile st = s_tile;
    const int32_t kvh = blockIdx.x % a.HKV;
    const int32_t len = st.end - st.begin;
    const int64_t row0 = (int64_t)st.tile * kRows;          // first row, of len * G
    const int64_t nrows = (int64_t)len * a.G;
    const int32_t last_token = (int32_t)(min(row0 + kRows, nrows) - 1) / a.G;
    const int32_t first_token = (int32_t)(row0 / a.G);

    // a tile of keys or values into the group's buffer
    auto bring = [&](float *to, int to_stride, const void *from, int64_t stride, int32_t k0) {
#pragma unroll
        for (int i = tid; i < kKeys * (D / 4); i += kGroup) {
            const int r = i / (D / 4), c = (i % (D / 4)) * 4;
            const bool in = k0 + r <= last_token;
            bring4(to + r * to_stride + c,
                   static_cast<const T *>(from) +
                       (in ? st.begin + (int64_t)k0 + r : st.begin) * stride + (int64_t)kvh * D + c,
                   in);
        }
        copies_issued();
    };
#pragma unroll
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        const bool in = row0 + r < nrows;
        const int64_t row = in ? row0 + r : 0;
        const int32_t tok = (int32_t)(row / a.G), h = (int32_t)(row % a.G);
        bring4(sq + r * KS + c,
               static_cast<const T *>(a.q) + (st.begin + (int64_t)tok) * a.q_stride +
                   ((int64_t)kvh * a.G + h) * D + c,
               in);
    }
    bring(sk, KS, a.k, a.k_stride, group * kKeys);
    int32_t tok[MI];  // token of each of the thread's rows (-1: no such row)
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t row = row0 + ty * MI + i;
        tok[i] = row < nrows ? (int32_t)(row / a.G) : -1;
    }
    const float c2 = a.scale * kLog2e;
    float m[MI], l[MI], acc[MI][CN][CW];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int n = 0; n < CN; ++n)
#pragma unroll
            for (int j = 0; j < CW; ++j) acc[i][n][j] = 0.f;
    }

    copies_landed<0>();
    __syncthreads();  // the queries
    for (int32_t k0 = group * kKeys; k0 <= last_token; k0 += GROUPS * kKeys) {
        copies_landed<0>();
        sync_group();  // the keys are there; the last tile's weights and values are done with
        bring(sv, D, a.v, a.v_stride, k0);
        // sums over the even and the odd channels, two to an instruction
        float2 s2[MI][4];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 qv[MI], kv[4];
#pragma unroll
            for (int i = 0; i < MI; ++i)
                qv[i] = *reinterpret_cast<const float4 *>(sq + (ty * MI + i) * KS + c);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                kv[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * KS + c);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s2[i][j] = f2_fma(make_float2(qv[i].x, qv[i].y),
                                      make_float2(kv[j].x, kv[j].y), s2[i][j]);
                    s2[i][j] = f2_fma(make_float2(qv[i].z, qv[i].w),
                                      make_float2(kv[j].z, kv[j].w), s2[i][j]);
                }
        }
        float s[MI][4];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
        const bool masked = k0 + kKeys - 1 > first_token;  // some key is past some row
        sync_group();  // the keys are done with
        if (kApart) bring(sk, KS, a.k, a.k_stride, k0 + GROUPS * kKeys);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (masked && k0 + tx + 16 * j > tok[i]) s[i][j] = -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // a row without keys so far keeps weights of 0 (and no NaN)
            const float ref = mx == -INFINITY ? 0.f : mx;
            const float corr = exp2f((m[i] - ref) * c2);
            m[i] = mx;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f((s[i][j] - ref) * c2);
                sp[(ty * MI + i) * kPStride + tx + 16 * j] = p;
                sum += p;
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[i] = l[i] * corr + sum;
#pragma unroll
            for (int n = 0; n < CN; ++n)
#pragma unroll
                for (int j = 0; j < CW; ++j) acc[i][n][j] *= corr;
        }
        copies_landed<kApart ? 1 : 0>();
        sync_group();
        auto weigh = [&](int kk, auto some_masked) {
            float4 pv[MI];
#pragma unroll
            for (int i = 0; i < MI; ++i)
                pv[i] = *reinterpret_cast<const float4 *>(sp + (ty * MI + i) * kPStride + kk);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float vv[CN][CW];
#pragma unroll
                for (int n = 0; n < CN; ++n) {
                    const float *src = sv + (kk + u) * D + n * 64 + tx * CW;
                    if constexpr (CW == 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(src);
                        vv[n][0] = x.x; vv[n][1] = x.y; vv[n][2] = x.z; vv[n][3] = x.w;
                    } else {
#pragma unroll
                        for (int j = 0; j < CW; ++j) vv[n][j] = src[j];
                    }
                }
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const float p = u == 0 ? pv[i].x : u == 1 ? pv[i].y : u == 2 ? pv[i].z : pv[i].w;
                    // a masked key adds nothing, whatever its value row holds
                    if (decltype(some_masked)::value && k0 + kk + u > tok[i]) continue;
#pragma unroll
                    for (int n = 0; n < CN; ++n) {
                        if constexpr (CW == 1) {
                            acc[i][n][0] = fmaf(p, vv[n][0], acc[i][n][0]);
                        } else {
#pragma unroll
                            for (int j = 0; j < CW; j += 2) {
                                const float2 y = f2_fma(make_float2(p, p),
                                                        make_float2(vv[n][j], vv[n][j + 1]),
                                                        make_float2(acc[i][n][j], acc[i][n][j + 1]));
                                acc[i][n][j] = y.x;
                                acc[i][n][j + 1] = y.y;
                            }
                        }
                    }
                }
            }
        };
        if (masked) {
            const int32_t kend = min(kKeys, last_token + 1 - k0);
            for (int kk = 0; kk < kend; kk += 4) weigh(kk, std::true_type{});
        } else {
#pragma unroll 4
            for (int kk = 0; kk < kKeys; kk += 4) weigh(kk, std::false_type{});
        }
        if (!kApart) {
            sync_group();
            bring(sk, KS, a.k, a.k_stride, k0 + GROUPS * kKeys);
        }
    }
    copies_landed<0>();
    if constexpr (GROUPS > 1) {
        // the other groups' states through the (now free) tiles: weighted
        // sums, maximum and sum of every row
        __syncthreads();
        if (group > 0) {
            float *mine = smem + (group - 1) * ROWS * (D + 2);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                float *r = mine + (ty * MI + i) * (D + 2);
                if (tx == 0) {
                    r[D] = m[i];
                    r[D + 1] = l[i];
                }
#pragma unroll
                for (int n = 0; n < CN; ++n)
#pragma unroll
                    for (int j = 0; j < CW; ++j) r[n * 64 + tx * CW + j] = acc[i][n][j];
            }
        }
        __syncthreads();
        if (group > 0) return;
        for (int g = 1; g < GROUPS; ++g)
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const float *r = smem + ((g - 1) * ROWS + ty * MI + i) * (D + 2);
                const float mx = fmaxf(m[i], r[D]), ref = mx == -INFINITY ? 0.f : mx;
                const float f0 = exp2f((m[i] - ref) * c2), f1 = exp2f((r[D] - ref) * c2);
                m[i] = mx;
                l[i] = l[i] * f0 + r[D + 1] * f1;
#pragma unroll
                for (int n = 0; n < CN; ++n)
#pragma unroll
                    for (int j = 0; j < CW; ++j)
                        acc[i][n][j] = acc[i][n][j] * f0 + r[n * 64 + tx * CW + j] * f1;
            }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        if (tok[i] < 0) continue;
        const int64_t row = row0 + ty * MI + i;
        const int64_t t = st.begin + (int64_t)tok[i];
        const int64_t head = (int64_t)kvh * a.G + row % a.G;
        const float inv = 1.f / l[i];
        if (a.lse && tx == 0) a.lse[t * a.HQ + head] = (m[i] * c2 + log2f(l[i])) * kLn2;
#pragma unroll
        for (int n = 0; n < CN; ++n)
#pragma unroll
            for (int j = 0; j < CW; ++j) {
                const int64_t o = (t * a.HQ + head) * D + n * 64 + tx * CW + j;
                const float y = acc[i][n][j] * inv;
                if (a.out_f32) static_cast<float *>(a.out)[o] = y;
                else static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(y);
            }
    }
}

template <typename T, int D, int ROWS, int GROUPS, int MI, int OCC>
cudaError_t launch_rows(const AttnArgs &a, cudaStream_t stream) {
    constexpr size_t bytes = smem_bytes<D, ROWS, GROUPS>();
    static_assert((GROUPS - 1) * ROWS * (D + 2) * sizeof(float) <= bytes, "the join fits");
    const cudaError_t e = allow_smem<attn_simt_kernel<T, D, ROWS, GROUPS, MI, OCC>>(bytes);
    if (e != cudaSuccess) return e;
    // every sequence's last tile may be short: at most N more than the rows fill
    const int64_t tiles = (int64_t)a.T * a.G / ROWS + a.N;
    attn_simt_kernel<T, D, ROWS, GROUPS, MI, OCC>
        <<<(unsigned)(tiles * a.HKV), GROUPS * ROWS / MI * 16, bytes, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t stream) {
    const int64_t tiles = ((int64_t)a.T * a.G / 64 + 1) * a.HKV;
    if (tiles < (int64_t)device_sms()) {
        // (D = 128: what shared memory holds)
        if constexpr (D == 128) return launch_rows<T, D, 32, 2, 4, 1>(a, stream);
        else return launch_rows<T, D, 16, 2, 4, 2>(a, stream);
    }
    if (a.T <= (int64_t)kKeys * a.N) return launch_rows<T, D, 64, 1, 4, 2>(a, stream);
    return launch_rows<T, D, 64, 2, 8, 1>(a, stream);
}

template <typename T>
cudaError_t launch_d(const AttnArgs &a, cudaStream_t stream) {
    switch (a.D) {
        case 16: return launch_t<T, 16>(a, stream);
        case 32: return launch_t<T, 32>(a, stream);
        case 64: return launch_t<T, 64>(a, stream);
        case 128: return launch_t<T, 128>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_attn_simt(const AttnArgs &a, cudaStream_t stream) {
    if (a.dtype == KDA_DTYPE_BF16) return launch_d<__nv_bfloat16>(a, stream);
    return launch_d<float>(a, stream);
}

}  // namespace kda

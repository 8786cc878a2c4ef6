// norm.hip -- root-mean-square norm over rows, with the residual's addition
// before it, an output in the storage type or in 8 bits, and its gradients.
//
//     t = x + res,  r = 1 / sqrt(mean(t^2) + eps),  y = t r w
//     8 bits:  scale = max(max|y| / 448, 2^-126),  out = e4m3(y / scale)
//     u = w dy:  dx = r (u - t r^2 mean(u t)) + dsum,   dw = sum over rows of dy t r
//
// All of it is fp32; t is rounded once for `sum` and not at all on its way to
// y, y once for out.  Bound by memory: a row is read once, held in registers
// by a wave or part of one, or by a workgroup.  16384 rows of 2560, bf16,
// a call on inputs that no cache holds: with residual and sum 66 us, 5.1 TB/s;
// with an 8-bit out instead 69 to 74 us, 4.0 to 4.3 TB/s; gradients with dsum 98
// to 103 us, 3.3 to 3.4 TB/s.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/fftconv.h"
#include "norm_ops.hpp"

namespace fftconv {
namespace {

template <typename T, int V> struct Piece { T v[V]; };
template <typename T, int V> __device__ __forceinline__ Piece<T, V> load(const T *p) {
    Piece<T, V> r;
    __builtin_memcpy(&r, __builtin_assume_aligned(p, V * sizeof(T)), sizeof r);
    return r;
}
// Results pass the caches by where they come in whole pieces of 16 bytes (16384 rows of 2560, bf16, sum and out: 65.5
// us, 71.3 with ordinary stores; 2048 rows of 4096: 13.2 and 13.6).
template <typename T, int V> __device__ __forceinline__ void store(T *p, const Piece<T, V> &r) {
    if constexpr (V * sizeof(T) == 16) {
        typedef uint32_t words __attribute__((ext_vector_type(4)));
        __builtin_nontemporal_store(__builtin_bit_cast(words, r), reinterpret_cast<words *>(p));
    } else {
        __builtin_memcpy(__builtin_assume_aligned(p, V * sizeof(T)), &r, sizeof r);
    }
}

// Sums (or largest bit patterns) over the LANES threads of a row, in all of them.  A row of 256 threads
// exchanges through `place`, which its caller does not write again before the next barrier but one.
template <int LANES> __device__ __forceinline__ float row_sum(float x, float *place) {
#pragma unroll
    for (int s = 1; s < (LANES < 64 ? LANES : 64); s <<= 1) x += __shfl_xor(x, s);
    if constexpr (LANES == 256) {
        if ((threadIdx.x & 63) == 0) place[threadIdx.x >> 6] = x;
        __syncthreads();
        x = (place[0] + place[1]) + (place[2] + place[3]);
    }
    return x;
}
template <int LANES> __device__ __forceinline__ uint32_t row_max(uint32_t x, uint32_t *place) {
#pragma unroll
    for (int s = 1; s < (LANES < 64 ? LANES : 64); s <<= 1) {
        const uint32_t o = __shfl_xor(x, s);
        x = o > x ? o : x;
    }
    if constexpr (LANES == 256) {
        if ((threadIdx.x & 63) == 0) place[threadIdx.x >> 6] = x;
        __syncthreads();
        const uint32_t a = place[0] > place[1] ? place[0] : place[1], b = place[2] > place[3] ? place[2] : place[3];
        x = a > b ? a : b;
    }
    return x;
}

__device__ __forceinline__ int64_t row_at(uint32_t row, uint32_t G, const int64_t (&s)[2]) {
    return G == 1 ? row * s[0] : (row / G) * s[0] + (row % G) * s[1];
}
__device__ __forceinline__ float inverse_rms(float squares, int D, float eps) { return 1.0f / sqrtf(squares / (float)D + eps); }

// V values as e4m3 (round to nearest even), y / scale of at most 448.  A product with the scale's rounded reciprocal lies
// beside some quotients that end in a tie of e4m3; what it leaves of y, times the reciprocal again, makes it the quotient
// rounded once.
template <int V> __device__ __forceinline__ void store8(uint8_t *p, const float (&from)[V], float scale, float inv) {
    const float whole = scale < __builtin_inff() ? scale : 0.0f;      // (an infinite scale leaves zeros and NaNs)
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float q = from[j] * inv;
        y[j] = __builtin_fmaf(__builtin_fmaf(-q, whole, from[j]), inv, q);
    }
    if constexpr (V % 4 == 0) {
        Piece<uint32_t, V / 4> r;
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            int u = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j], y[4 * j + 1], 0, false);
            r.v[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j + 2], y[4 * j + 3], u, true);
        }
        store<uint32_t, V / 4>(reinterpret_cast<uint32_t *>(p), r);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[j], 0.0f, 0, false);
    }
}

// LANES threads a row, NV pieces of V values each; NV = 0: any width, the row's values read again for
// every pass over them.
template <typename T, int V, int LANES, int NV, bool EIGHT>
__global__ __launch_bounds__(256) void norm_fwd_kernel(const NormFwd a) {
    constexpr uint32_t R = 256 / LANES;
    constexpr int HELD = NV ? NV : 1;
    __shared__ float place[2][4];
    __shared__ uint32_t place_max[2][4];
    const int lane = threadIdx.x % LANES;
    const int pieces = (a.D + V - 1) / V;      // (V divides D)
    int turn = 0;
    // rows of one workgroup are neighbours; all threads of a workgroup run the same rounds
    for (uint32_t row0 = blockIdx.x * R; row0 < a.rows; row0 += gridDim.x * R, turn ^= 1) {
        const uint32_t row = row0 + threadIdx.x / LANES;
        const bool live = row < a.rows;
        const uint32_t at = live ? row : a.rows - 1;
        const T *x = static_cast<const T *>(a.x) + row_at(at, a.G, a.xs);
        const T *res = a.res ? static_cast<const T *>(a.res) + row_at(at, a.G, a.rs) : nullptr;
        T *sum = a.sum ? static_cast<T *>(a.sum) + row_at(at, a.G, a.ss) : nullptr;
        auto values = [&](int i, float (&t)[V]) __attribute__((always_inline)) {
            const Piece<T, V> p = load<T, V>(x + i * V);
#pragma unroll
            for (int j = 0; j < V; ++j) t[j] = (float)p.v[j];
            if (res) {
                const Piece<T, V> q = load<T, V>(res + i * V);
#pragma unroll
                for (int j = 0; j < V; ++j) t[j] += (float)q.v[j];
            }
        };
        float t[HELD][V], squares = 0.0f;
        if constexpr (NV > 0) {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int i = n * LANES + lane;
                if (i < pieces) values(i, t[n]);
                else
#pragma unroll
                    for (int j = 0; j < V; ++j) t[n][j] = 0.0f;
            }
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int j = 0; j < V; ++j) squares += t[n][j] * t[n][j];
        } else {
            for (int i = lane; i < pieces; i += LANES) {
                values(i, t[0]);
#pragma unroll
                for (int j = 0; j < V; ++j) squares += t[0][j] * t[0][j];
            }
        }
        const float r = inverse_rms(row_sum<LANES>(squares, place[turn]), a.D, a.eps);
        const T *w = static_cast<const T *>(a.weight);
        auto normed = [&](int i, const float (&from)[V], float (&y)[V]) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = from[j] * r;
            if (w) {
                const Piece<T, V> p = load<T, V>(w + i * V);
#pragma unroll
                for (int j = 0; j < V; ++j) y[j] *= (float)p.v[j];
            }
        };
        auto keep = [&](int i, const float (&from)[V]) __attribute__((always_inline)) {
            if (!sum) return;
            Piece<T, V> p;
#pragma unroll
            for (int j = 0; j < V; ++j) p.v[j] = (T)from[j];
            store<T, V>(sum + i * V, p);
        };
        // pieces in turn, from registers or memory; sum (which may lie on res or x) is written last of all reads
        auto each = [&](auto &&f) __attribute__((always_inline)) {
            if constexpr (NV > 0) {
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int i = n * LANES + lane;
                    if (live & (i < pieces)) f(i, t[n]);
                }
            } else {
                for (int i = lane; i < pieces; i += LANES) {
                    values(i, t[0]);
                    if (live) f(i, t[0]);
                }
            }
        };
        if constexpr (EIGHT) {
            uint32_t top = 0;
            each([&](int i, float (&from)[V]) __attribute__((always_inline)) {
                float y[V];
                normed(i, from, y);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const uint32_t u = __builtin_bit_cast(uint32_t, y[j]) & 0x7fffffffu;   // a NaN counts as the largest
                    top = u > top ? u : top;
                }
            });
            const float most = __builtin_bit_cast(float, row_max<LANES>(top, place_max[turn])) / 448.0f;
            const float scale = most < 0x1p-126f ? 0x1p-126f : most;
            const float inv = 1.0f / scale;
            if (live && lane == 0) a.scales[row] = scale;
            uint8_t *o = static_cast<uint8_t *>(a.out) + row_at(at, a.G, a.os);
            each([&](int i, float (&from)[V]) __attribute__((always_inline)) {
                float y[V];
                normed(i, from, y);
                store8<V>(o + i * V, y, scale, inv);
                keep(i, from);
            });
        } else {
            T *o = static_cast<T *>(a.out) + row_at(at, a.G, a.os);
            each([&](int i, float (&from)[V]) __attribute__((always_inline)) {
                float y[V];
                normed(i, from, y);
                Piece<T, V> p;
#pragma unroll
                for (int j = 0; j < V; ++j) p.v[j] = (T)y[j];
                store<T, V>(o + i * V, p);
                keep(i, from);
            });
        }
    }
}

// Rows held in registers: dx, and each workgroup's own sums of the weight's gradient.
template <typename T, int V, int LANES, int NV>
__global__ __launch_bounds__(256) void norm_bwd_kernel(const NormBwd a) {
    constexpr uint32_t R = 256 / LANES;
    __shared__ float place[2][2][4];
    __shared__ float joined[LANES < 256 ? LANES * NV * V : 1];
    const int lane = threadIdx.x % LANES;
    const int pieces = a.D / V;
    const T *weight = static_cast<const T *>(a.weight);
    float dw[NV][V];
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[n][j] = 0.0f;
    int turn = 0;
    for (uint32_t row0 = blockIdx.x * R; row0 < a.rows; row0 += gridDim.x * R, turn ^= 1) {
        const uint32_t row = row0 + threadIdx.x / LANES;
        const bool live = row < a.rows;
        const uint32_t at = live ? row : a.rows - 1;
        const T *x = static_cast<const T *>(a.x) + row_at(at, a.G, a.xs);
        const T *dy = static_cast<const T *>(a.dout) + row_at(at, a.G, a.gs);
        Piece<T, V> xv[NV], gv[NV];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int i = n * LANES + lane;
            if (live & (i < pieces)) {
                xv[n] = load<T, V>(x + i * V);
                gv[n] = load<T, V>(dy + i * V);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) xv[n].v[j] = gv[n].v[j] = (T)0.0f;
            }
        }
        float squares = 0.0f, along = 0.0f;
        float u[NV][V];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int i = n * LANES + lane;
#pragma unroll
            for (int j = 0; j < V; ++j) u[n][j] = (float)gv[n].v[j];
            if (weight && i < pieces) {
                const Piece<T, V> p = load<T, V>(weight + i * V);
#pragma unroll
                for (int j = 0; j < V; ++j) u[n][j] *= (float)p.v[j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float t = (float)xv[n].v[j];
                squares += t * t;
                along += u[n][j] * t;
            }
        }
        const float r = inverse_rms(row_sum<LANES>(squares, place[turn][0]), a.D, a.eps);
        const float c = row_sum<LANES>(along, place[turn][1]) / (float)a.D * r * r;
        T *dx = a.dx ? static_cast<T *>(a.dx) + row_at(at, a.G, a.ds) : nullptr;
        const T *more = a.dsum ? static_cast<const T *>(a.dsum) + row_at(at, a.G, a.us) : nullptr;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int i = n * LANES + lane;
            if (live) {      // (a row beyond the last may have r = inf)
#pragma unroll
                for (int j = 0; j < V; ++j) dw[n][j] += (float)gv[n].v[j] * ((float)xv[n].v[j] * r);
            }
            if (live & (i < pieces) & (dx != nullptr)) {
                float d[V];
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = r * (u[n][j] - (float)xv[n].v[j] * c);
                if (more) {
                    const Piece<T, V> p = load<T, V>(more + i * V);
#pragma unroll
                    for (int j = 0; j < V; ++j) d[j] += (float)p.v[j];
                }
                Piece<T, V> p;
#pragma unroll
                for (int j = 0; j < V; ++j) p.v[j] = (T)d[j];
                store<T, V>(dx + i * V, p);
            }
        }
    }
    if (!a.part) return;
    float *part = a.part + (int64_t)blockIdx.x * a.D;
    if constexpr (LANES == 256) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int i = n * LANES + lane;
            if (i < pieces)
#pragma unroll
                for (int j = 0; j < V; ++j) part[i * V + j] = dw[n][j];
        }
    } else {
        // the workgroup's rows one after another, so that the sum has one order
        for (uint32_t g = 0; g < R; ++g) {
            if (threadIdx.x / LANES == g)
#pragma unroll
                for (int n = 0; n < NV; ++n)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float &s = joined[(n * V + j) * LANES + lane];
                        s = g == 0 ? dw[n][j] : s + dw[n][j];
                    }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < a.D; i += 256) {
            const int piece = i / V, j = i % V;
            part[i] = joined[(piece / LANES * V + j) * LANES + piece % LANES];
        }
    }
}

// Rows too wide for a workgroup's registers: r and the factor of t first, then slabs of rows by columns.
template <typename T, int V> __global__ __launch_bounds__(256) void norm_bwd_stats_kernel(const NormBwd a) {
    __shared__ float place[2][2][4];
    const int pieces = a.D / V;
    const T *weight = static_cast<const T *>(a.weight);
    int turn = 0;
    for (uint32_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T *x = static_cast<const T *>(a.x) + row_at(row, a.G, a.xs);
        const T *dy = static_cast<const T *>(a.dout) + row_at(row, a.G, a.gs);
        float squares = 0.0f, along = 0.0f;
        for (int i = threadIdx.x; i < pieces; i += 256) {
            const Piece<T, V> xv = load<T, V>(x + (int64_t)i * V), gv = load<T, V>(dy + (int64_t)i * V);
            Piece<T, V> wv;
            if (weight) wv = load<T, V>(weight + (int64_t)i * V);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float t = (float)xv.v[j], u = weight ? (float)gv.v[j] * (float)wv.v[j] : (float)gv.v[j];
                squares += t * t;
                along += u * t;
            }
        }
        const float r = inverse_rms(row_sum<256>(squares, place[turn][0]), a.D, a.eps);
        const float c = row_sum<256>(along, place[turn][1]) / (float)a.D * r * r;
        if (threadIdx.x == 0) {
            a.stats[2 * (int64_t)row] = r;
            a.stats[2 * (int64_t)row + 1] = c;
        }
    }
}
// grid (column pieces / 256, slabs)
template <typename T, int V> __global__ __launch_bounds__(256) void norm_bwd_wide_kernel(const NormBwd a) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.D / V) return;
    const T *weight = static_cast<const T *>(a.weight);
    float w[V], dw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = 1.0f, dw[j] = 0.0f;
    if (weight) {
        const Piece<T, V> p = load<T, V>(weight + (int64_t)i * V);
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = (float)p.v[j];
    }
    for (uint32_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const Piece<T, V> xv = load<T, V>(static_cast<const T *>(a.x) + row_at(row, a.G, a.xs) + (int64_t)i * V);
        const Piece<T, V> gv = load<T, V>(static_cast<const T *>(a.dout) + row_at(row, a.G, a.gs) + (int64_t)i * V);
        const float r = a.stats[2 * (int64_t)row], c = a.stats[2 * (int64_t)row + 1];
        float d[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float t = (float)xv.v[j], g = (float)gv.v[j];
            dw[j] += g * (t * r);
            d[j] = r * (g * w[j] - t * c);
        }
        if (!a.dx) continue;
        if (a.dsum) {
            const Piece<T, V> p = load<T, V>(static_cast<const T *>(a.dsum) + row_at(row, a.G, a.us) + (int64_t)i * V);
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] += (float)p.v[j];
        }
        Piece<T, V> p;
#pragma unroll
        for (int j = 0; j < V; ++j) p.v[j] = (T)d[j];
        store<T, V>(static_cast<T *>(a.dx) + row_at(row, a.G, a.ds) + (int64_t)i * V, p);
    }
    if (a.part)
#pragma unroll
        for (int j = 0; j < V; ++j) a.part[(int64_t)blockIdx.y * a.D + (int64_t)i * V + j] = dw[j];
}

// dweight <- sums of the slabs' parts, in one order: 16 threads of a column take the slabs in turn.
template <typename T> __global__ __launch_bounds__(256) void norm_join_kernel(const float *part, int64_t slabs, int D, T *dweight) {
    __shared__ float own[16][17];
    const int c = threadIdx.x & 15, s0 = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
    float sum = 0.0f;
    if (col < D)
        for (int64_t s = s0; s < slabs; s += 16) sum += part[s * D + col];
    own[s0][c] = sum;
    __syncthreads();
    if (s0 == 0 && col < D) {
#pragma unroll
        for (int i = 1; i < 16; ++i) sum += own[i][c];
        dweight[col] = (T)sum;
    }
}

template <int MOST, typename F> hipError_t with_loads(int loads, F &&f) {
    if (loads == MOST) return f(std::integral_constant<int, MOST>{});
    if constexpr (MOST > 1) return with_loads<MOST - 1>(loads, f);
    return hipErrorInvalidValue;
}
// lanes: 8, 16 or 32 with one piece each, 64 with up to WAVE, 256 with up to eight
template <int WAVE, typename F> hipError_t with_lanes(const NormPlan &p, F &&f) {
    if (p.lanes == 8 && p.loads == 1) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
    if (p.lanes == 16 && p.loads == 1) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    if (p.lanes == 32 && p.loads == 1) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
    if (p.lanes == 64)
        return with_loads<WAVE>(p.loads, [&](auto n) { return f(std::integral_constant<int, 64>{}, n); });
    if (p.lanes == 256)
        return with_loads<8>(p.loads, [&](auto n) { return f(std::integral_constant<int, 256>{}, n); });
    return hipErrorInvalidValue;
}

template <typename T, int V> hipError_t fwd_vec(const NormFwd &a, const NormPlan &p, hipStream_t s) {
    const unsigned grid = (unsigned)p.groups;
    if (p.loads == 0) {
        if (a.scales) norm_fwd_kernel<T, V, 256, 0, true><<<grid, 256, 0, s>>>(a);
        else norm_fwd_kernel<T, V, 256, 0, false><<<grid, 256, 0, s>>>(a);
        return hipGetLastError();
    }
    return with_lanes<kFwdWave>(p, [&](auto lanes, auto loads) {
        if (a.scales) norm_fwd_kernel<T, V, decltype(lanes)::value, decltype(loads)::value, true><<<grid, 256, 0, s>>>(a);
        else norm_fwd_kernel<T, V, decltype(lanes)::value, decltype(loads)::value, false><<<grid, 256, 0, s>>>(a);
        return hipGetLastError();
    });
}
template <typename T, int V> hipError_t bwd_vec(const NormBwd &a, const NormPlan &p, void *dweight, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (a.rows > 0) {
        if (p.loads == 0) {
            norm_bwd_stats_kernel<T, V><<<(unsigned)p.groups, 256, 0, s>>>(a);
            norm_bwd_wide_kernel<T, V><<<dim3((unsigned)((a.D / V + 255) / 256), (unsigned)p.slabs), 256, 0, s>>>(a);
            e = hipGetLastError();
        } else {
            e = with_lanes<kBwdWave>(p, [&](auto lanes, auto loads) {
                norm_bwd_kernel<T, V, decltype(lanes)::value, decltype(loads)::value><<<(unsigned)p.groups, 256, 0, s>>>(a);
                return hipGetLastError();
            });
        }
    }
    if (e == hipSuccess && dweight) {
        norm_join_kernel<T><<<(unsigned)((a.D + 15) / 16), 256, 0, s>>>(a.part, a.rows > 0 ? p.slabs : 0, a.D, static_cast<T *>(dweight));
        e = hipGetLastError();
    }
    return e;
}

}  // namespace

hipError_t launch_norm_fwd(int dtype, const NormFwd &a, const NormPlan &p, hipStream_t s) {
    if (dtype == FFTCONV_F32) return p.vec == 4 ? fwd_vec<float, 4>(a, p, s) : fwd_vec<float, 1>(a, p, s);
    if (dtype == FFTCONV_F16) return p.vec == 8 ? fwd_vec<_Float16, 8>(a, p, s) : fwd_vec<_Float16, 1>(a, p, s);
    return p.vec == 8 ? fwd_vec<__bf16, 8>(a, p, s) : fwd_vec<__bf16, 1>(a, p, s);
}
hipError_t launch_norm_bwd(int dtype, const NormBwd &a, const NormPlan &p, void *dweight, hipStream_t s) {
    if (dtype == FFTCONV_F32) return p.vec == 4 ? bwd_vec<float, 4>(a, p, dweight, s) : bwd_vec<float, 1>(a, p, dweight, s);
    if (dtype == FFTCONV_F16) return p.vec == 8 ? bwd_vec<_Float16, 8>(a, p, dweight, s) : bwd_vec<_Float16, 1>(a, p, dweight, s);
    return p.vec == 8 ? bwd_vec<__bf16, 8>(a, p, dweight, s) : bwd_vec<__bf16, 1>(a, p, dweight, s);
}

}  // namespace fftconv

// pn_norm.hip - what stands between two blocks of a decoder
// (pn_residual_norm), for AMD Instinct MI355X (gfx950).
//
//   u  = y, or y * post_gain / sqrt(mean(y^2) + eps)
//   h' = h + scale * chan_scale * gate(z) * u
//   x  = fp16(h' * pre_gain / sqrt(mean(h'^2) + eps))
//
// One pass: a row's h, y and z are loaded at once into registers and stay
// there; the two means are the only things its threads wait for each other
// for.  Everything is fp32, rounded once where it is written; sums of squares
// run per thread, then over the wave and the waves in a fixed order.
//
// What bounds it: memory in large calls, 8191 rows of 5120 with a gate (755 MB)
// 136 us, 5.5 TB/s; a launch and the reductions in small ones, 512 rows 7.6 us,
// one row 3.8.
#include "pn_device.h"
#include "pn_kv4.h"

using namespace pn;
using namespace pn::host;

namespace {

typedef float float4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

struct NormArgs {
    const float *h, *post_gain, *chan_scale, *pre_gain;
    const void *y, *z;
    float *h_out;
    uint16_t *x;
    int64_t ldh, ldy, ldz, ldho, ldx, T;
    int32_t n, post, gate;
    float scale, eps, inv_n;
};

// Four elements from i on of a row of n; elements past it are `rest`.
template <typename T4, typename T>
__device__ __forceinline__ float4_t load4(const T *row, int i, int n, float rest)
{
    if (i + 4 <= n) {
        const T4 v = *(const T4 *)(row + i);
        return (float4_t){(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
    }
    float4_t v = {rest, rest, rest, rest};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (i + e < n) v[e] = (float)row[i + e];
    return v;
}

template <bool HALF> __device__ __forceinline__ float4_t load_rows(const void *row, int i, int n)
{
    if constexpr (HALF) return load4<half4_t>((const _Float16 *)row, i, n, 0.0f);
    else return load4<float4_t>((const float *)row, i, n, 0.0f);
}

// 1 / (1 + exp(-z)).  The product z log2(e) is kept to twice its precision,
// as exp2 turns its rounding into one of |z| steps; the reciprocal is refined
// once.  Beyond 88 the result stays 1, below -88 it is under 2^-126.
__device__ __forceinline__ float sigmoid(float z)
{
    z = z < -88.0f ? -88.0f : z > 88.0f ? 88.0f : z;  // a NaN stays
    const float hi = z * -1.44269502162933349609375f;
    const float lo = __builtin_fmaf(z, -1.92596299112661746887e-8f, __builtin_fmaf(z, -1.44269502162933349609375f, -hi));
    float e = __builtin_amdgcn_exp2f(hi);
    e = __builtin_fmaf(e, lo * 0.693147180559945f, e);
    const float d = 1.0f + e, r = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}
// z / (1 + exp(-z)); 0 at -inf, where the product would be NaN.
__device__ __forceinline__ float silu(float z) { return (z < -88.0f ? -88.0f : z) * sigmoid(z); }

// Sum over a row's threads: W waves, in every one of them.
template <int W> __device__ __forceinline__ float row_sum(float v, float *part)
{
    v = wave_sum(v);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w];
    }
    return v;
}

// W waves a row, V groups of four elements a thread; with W = 1 four rows a
// workgroup.
template <int W, int V, bool HALF>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void residual_norm(NormArgs a)
{
    __shared__ float part[2][W];
    const int tid = W == 1 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int64_t t = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
    if (t >= a.T) return;  // W = 1 alone, where no wave waits for another
    const int n = a.n;
    const float *h_row = a.h + t * a.ldh;
    const uint8_t *y_row = (const uint8_t *)a.y + t * a.ldy * (HALF ? 2 : 4);
    const uint8_t *z_row = (const uint8_t *)a.z + t * a.ldz * (HALF ? 2 : 4);
    float4_t h[V], u[V], z[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = 4 * (tid + 64 * W * i);
        h[i] = u[i] = z[i] = (float4_t){0, 0, 0, 0};
        if (at < n) {
            h[i] = load4<float4_t>(h_row, at, n, 0.0f);
            if (a.y) u[i] = load_rows<HALF>(y_row, at, n);
            if (a.gate) z[i] = load_rows<HALF>(z_row, at, n);
        }
    }
    if (a.y) {
        float r = 1.0f;
        if (a.post) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s = __builtin_fmaf(u[i][e], u[i][e], s);
            r = 1.0f / __builtin_sqrtf(row_sum<W>(s, part[0]) * a.inv_n + a.eps);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = 4 * (tid + 64 * W * i);
            if (at >= n) continue;
            float4_t f = {a.scale, a.scale, a.scale, a.scale};
            if (a.chan_scale) f *= load4<float4_t>(a.chan_scale, at, n, 0.0f);
            if (a.post) f *= r;
            if (a.post_gain) f *= load4<float4_t>(a.post_gain, at, n, 0.0f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float g = 1.0f;
                if (a.gate == PN_GATE_PLAIN) g = z[i][e];
                else if (a.gate == PN_GATE_SIGMOID) g = sigmoid(z[i][e]);
                else if (a.gate == PN_GATE_SILU) g = silu(z[i][e]);
                h[i][e] = __builtin_fmaf(f[e] * g, u[i][e], h[i][e]);
            }
        }
    }
    if (a.h_out) {
        float *row = a.h_out + t * a.ldho;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = 4 * (tid + 64 * W * i);
            if (at + 4 <= n) {
                // read again a whole block later: past the caches (8191 rows of 5120 145 -> 141 us)
                __builtin_nontemporal_store(h[i], (float4_t *)(row + at));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (at + e < n) row[at + e] = h[i][e];
            }
        }
    }
    if (!a.x) return;  // the whole launch
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = __builtin_fmaf(h[i][e], h[i][e], s);
    const float r = 1.0f / __builtin_sqrtf(row_sum<W>(s, part[1]) * a.inv_n + a.eps);
    uint16_t *row = a.x + t * a.ldx;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = 4 * (tid + 64 * W * i);
        if (at >= n) continue;
        float4_t v = h[i] * r;
        if (a.pre_gain) v *= load4<float4_t>(a.pre_gain, at, n, 0.0f);
        const half4_t w = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
        if (at + 4 <= n) {
            *(half4_t *)(row + at) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at + e < n) ((_Float16 *)row)[at + e] = w[e];
        }
    }
}

// A launch holds less than 2^32 threads; further rows go into further ones.
template <int W, int V, bool HALF> pn_status launch(NormArgs a, hipStream_t s)
{
    constexpr int kThreads = W == 1 ? 256 : 64 * W, kRows = W == 1 ? 4 : 1, kBytes = HALF ? 2 : 4;
    constexpr int64_t kMost = (int64_t)UINT32_MAX / kThreads * kRows;
    const int64_t all = a.T;
    for (int64_t t = 0; t < all; t += kMost) {
        a.T = all - t < kMost ? all - t : kMost;
        const unsigned blocks = (unsigned)((a.T + kRows - 1) / kRows);
        hipLaunchKernelGGL((residual_norm<W, V, HALF>), dim3(blocks), dim3(kThreads), 0, s, a);
        if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
        a.h += kMost * a.ldh;
        if (a.y) a.y = (const uint8_t *)a.y + kMost * a.ldy * kBytes;
        if (a.z) a.z = (const uint8_t *)a.z + kMost * a.ldz * kBytes;
        if (a.h_out) a.h_out += kMost * a.ldho;
        if (a.x) a.x += kMost * a.ldx;
    }
    return PN_OK;
}

template <int W, int V, int MAX, bool HALF> pn_status pick(const NormArgs &a, int v, hipStream_t s)
{
    if constexpr (V < MAX) {
        if (v > V) return pick<W, V + 1, MAX, HALF>(a, v, s);
    }
    return launch<W, V, HALF>(a, s);
}

// A row's waves: as few as hold it in registers with a few groups a thread.
// More share the reductions' latency but leave fewer rows at work: 512 rows of
// 5120: 4 waves 9.7 us, 8 waves 8.0, 16 waves 7.8; 8191 rows with a gate 145,
// 141, 142; 3001 rows of 1027: 1 wave 14.3 us, 2 waves 12.9, 4 waves 14.3.
template <bool HALF> pn_status run(const NormArgs &a, hipStream_t s)
{
    const int groups = (a.n + 3) / 4;
    if (groups <= 256) return pick<1, 1, 4, HALF>(a, (groups + 63) / 64, s);
    if (groups <= 512) return pick<2, 3, 4, HALF>(a, (groups + 127) / 128, s);
    if (groups <= 2048) return pick<8, 2, 4, HALF>(a, (groups + 511) / 512, s);
    return pick<16, 3, 8, HALF>(a, (groups + 1023) / 1024, s);
}

}  // namespace

extern "C" pn_status pn_residual_norm(const pn_residual_norm_desc *d, void *stream)
{
    if (!d || !d->h || (!d->h_out && !d->x)) return PN_EINVAL;
    if ((d->row_type != PN_ROWS_F32 && d->row_type != PN_ROWS_F16) || d->gate < PN_GATE_NONE || d->gate > PN_GATE_SILU)
        return PN_EINVAL;
    if ((d->gate != PN_GATE_NONE) != (d->z != nullptr)) return PN_EINVAL;
    if (!d->y && (d->z || d->post || d->post_gain || d->chan_scale)) return PN_EINVAL;
    if (d->post_gain && !d->post) return PN_EINVAL;
    if (d->T < 0 || d->n < 1) return PN_ESHAPE;
    if (!(__builtin_fabsf(d->scale) <= 0x1.fffffep127f) || !(d->eps >= 0.0f && d->eps <= 0x1.fffffep127f)) return PN_ESHAPE;
    const int64_t n = d->n;
    if (d->ldh < n || (d->y && d->ldy < n) || (d->z && d->ldz != 0 && d->ldz < n) || (d->h_out && d->ldho < n) ||
        (d->x && d->ldx < n))
        return PN_ESHAPE;
    const int step = d->row_type == PN_ROWS_F16 ? 8 : 4, bytes = d->row_type == PN_ROWS_F16 ? 2 : 4;
    const void *arrays[] = {d->h, d->y, d->z, d->h_out, d->x, d->post_gain, d->chan_scale, d->pre_gain};
    for (const void *p : arrays)
        if (!aligned(p, 16)) return PN_EALIGN;
    if (d->ldh % 4 || (d->y && d->ldy % step) || (d->z && d->ldz % step) || (d->h_out && d->ldho % 4) || (d->x && d->ldx % 8))
        return PN_EALIGN;
    if (n > PN_NORM_MAX || d->T > INT32_MAX) return PN_EUNSUPPORTED;
    if (d->T == 0) return PN_OK;
    const int64_t T = d->T;
    const Rows h = {d->h, d->ldh * 4, n * 4, T}, y = {d->y, d->ldy * bytes, n * bytes, T};
    const Rows z = {d->z, d->ldz * bytes, n * bytes, d->ldz ? T : 1}, ho = {d->h_out, d->ldho * 4, n * 4, T};
    const Rows x = {d->x, d->ldx * 2, n * 2, T};
    const Rows inputs[] = {y, z, {d->post_gain, 0, n * 4, 1}, {d->chan_scale, 0, n * 4, 1}, {d->pre_gain, 0, n * 4, 1}};
    for (const Rows &r : inputs)
        if (overlap(r, ho) || overlap(r, x)) return PN_EINVAL;
    const bool in_place = d->h_out == d->h && d->ldho == d->ldh;
    if ((!in_place && overlap(h, ho)) || overlap(h, x) || overlap(ho, x)) return PN_EINVAL;

    NormArgs a;
    a.h = d->h;
    a.post_gain = d->post_gain;
    a.chan_scale = d->chan_scale;
    a.pre_gain = d->pre_gain;
    a.y = d->y;
    a.z = d->z;
    a.h_out = in_place && !d->y ? nullptr : d->h_out;  // nothing changes
    a.x = d->x;
    a.ldh = d->ldh;
    a.ldy = d->ldy;
    a.ldz = d->ldz;
    a.ldho = d->ldho;
    a.ldx = d->ldx;
    a.T = T;
    a.n = (int32_t)n;
    a.post = d->post != 0;
    a.gate = d->gate;
    a.scale = d->scale;
    a.eps = d->eps;
    a.inv_n = (float)(1.0 / (double)n);
    const hipStream_t s = (hipStream_t)stream;
    const pn_status st = bytes == 2 ? run<true>(a, s) : run<false>(a, s);
    if (st == PN_OK) g_last_variant = kVarResidualNorm;
    return st;
}

// pn_spec.hip - verification of drafted tokens against the target's
// probabilities (pn_spec_verify), for AMD Instinct MI355X (gfx950).
//
// Draft j of a request is accepted while u_j q_j(x_j) < p_j(x_j); products of
// two fp32 numbers are exact in fp64, so the comparison is the exact one.
// One more token is drawn from the row after the last accepted draft, from
// r = max(p - q, 0) or from p: the first index whose inclusive prefix sum is
// above u_k * sum r.  The difference of two fp32 numbers is rounded once, as
// fp32; the sums run in fp64, where a row of 2^18 entries leaves 2^-35 of the
// total, so their grouping does not move a border that fp32 inputs can show.
//
// Only one target row and one draft row of each request are read whole: the
// bytes are B * V * 8.  Kernel spec_sums cuts a row into chunks, one
// workgroup a chunk with all of its loads in flight at once, and leaves each
// chunk's sum of r and of p (which serves where nothing of r is left); every
// workgroup finds the row by itself from the few gathered probabilities, and
// the first chunk's notes how many drafts stand.  Kernel spec_pick, one
// workgroup a request, finds the chunk that holds the border from the sums
// (every wave for itself), then the index within it: two rounds of loads and
// two barriers, because with few requests latency is all there is.  A
// workgroup of one launch never waits for another.
//
// 64 requests of 248320 entries: sums 20 us, 6.1 TB/s, of 6.9 that streaming
// reads reach here; pick 8.0.  One request of 62080: 4.3 and 7.2, launches
// and a chain of dependent loads.
#include "pn_kv4.h"

using namespace pn::host;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kChunk = 4096;  // entries of a chunk

struct SpecArgs {
    const float *target, *draft, *u;
    const int32_t *tokens, *n_draft;
    int32_t *out, *accepted;
    double *sums;  // [B][chunks][2]: of r, of p
    int32_t *took; // [B]: drafts that stand
    int64_t ldt, ldd, ld_tok, ldu, ld_out, V;
    int32_t k, chunks;
};

// Only positive finite entries count.
__device__ __forceinline__ float clean(float v) { return v > 0.0f && v < __builtin_inff() ? v : 0.0f; }

// The row a request draws from.
struct Row {
    const float *p;  // target row
    const float *q;  // draft row, or NULL
    int32_t drop;    // index whose r is 0 (no draft probabilities), or -1
    int32_t accepted;
    __device__ __forceinline__ float r(int64_t i) const
    {
        float v = p[i];
        if (q) v -= q[i];
        return i == drop ? 0.0f : clean(v);
    }
};

// Drafts of request b that are tested.
__device__ __forceinline__ int drafts(const SpecArgs &a, int b)
{
    const int n = a.n_draft ? a.n_draft[b] : a.k;
    return n < 0 ? 0 : n > a.k ? a.k : n;
}

// How many of them stand.  Every wave computes this alike: lane j tests draft j.
__device__ __forceinline__ int standing(const SpecArgs &a, int b, int n, int lane)
{
    for (int j0 = 0; j0 < n; j0 += 64) {
        const int j = j0 + lane;
        bool ok = true;
        if (j < n) {
            const int32_t x = a.tokens[b * a.ld_tok + j];
            ok = false;
            if (x >= 0 && x < a.V) {
                const double p = a.target[((int64_t)b * (a.k + 1) + j) * a.ldt + x];
                const double q = a.draft ? (double)a.draft[((int64_t)b * a.k + j) * a.ldd + x] : 1.0;
                ok = (double)a.u[b * a.ldu + j] * q < p;
            }
        }
        const uint64_t bad = __ballot(!ok);
        if (bad) return j0 + __builtin_ctzll(bad);
    }
    return n;
}

// The row that a request with `took` of n drafts standing draws from.
__device__ __forceinline__ Row row_of(const SpecArgs &a, int b, int n, int took)
{
    Row row;
    row.accepted = took;
    row.p = a.target + ((int64_t)b * (a.k + 1) + took) * a.ldt;
    row.q = took < n && a.draft ? a.draft + ((int64_t)b * a.k + took) * a.ldd : nullptr;
    row.drop = took < n && !a.draft ? a.tokens[b * a.ld_tok + took] : -1;
    return row;
}

// Four entries at once from a row that need only be aligned to one.
typedef float float4_a4 __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kEach = kChunk / kThreads;  // entries of a thread

__global__ __launch_bounds__(kThreads) void spec_sums(SpecArgs a)
{
    __shared__ double part[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.y;
    const int n = drafts(a, b);
    const Row row = row_of(a, b, n, standing(a, b, n, lane));
    const int64_t lo = (int64_t)blockIdx.x * kChunk, hi = lo + kChunk < a.V ? lo + kChunk : a.V;
    double sr = 0.0, sp = 0.0;
    if (hi - lo == kChunk) {
        float4_a4 p[kEach / 4], q[kEach / 4] = {};
#pragma unroll
        for (int i = 0; i < kEach / 4; ++i) p[i] = *(const float4_a4 *)(row.p + lo + 4 * (threadIdx.x + kThreads * i));
        if (row.q) {
#pragma unroll
            for (int i = 0; i < kEach / 4; ++i) q[i] = *(const float4_a4 *)(row.q + lo + 4 * (threadIdx.x + kThreads * i));
        }
#pragma unroll
        for (int i = 0; i < kEach / 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool drop = lo + 4 * (threadIdx.x + kThreads * i) + e == row.drop;
                sr += drop ? 0.0 : (double)clean(row.q ? p[i][e] - q[i][e] : p[i][e]);
                sp += (double)clean(p[i][e]);
            }
    } else {
        for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
            sr += (double)row.r(i);
            sp += (double)clean(row.p[i]);
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        sr += __shfl_xor(sr, d, 64);
        sp += __shfl_xor(sp, d, 64);
    }
    __shared__ double part_p[kWaves];
    if (lane == 0) part[wave] = sr, part_p[wave] = sp;
    __syncthreads();
    if (threadIdx.x == 0) {
        sr = sp = 0.0;
        for (int w = 0; w < kWaves; ++w) sr += part[w], sp += part_p[w];
        double *s = a.sums + 2 * ((int64_t)b * a.chunks + blockIdx.x);
        s[0] = sr;
        s[1] = sp;
        if (blockIdx.x == 0) a.took[b] = row.accepted;
    }
}

// Inclusive prefix over the wave.
__device__ __forceinline__ double wave_prefix(double x, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    return x;
}

__global__ __launch_bounds__(kThreads) void spec_pick(SpecArgs a)
{
    __shared__ double part[kWaves];
    __shared__ int32_t found, last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x;
    const double *s = a.sums + 2 * (int64_t)b * a.chunks;
    const int n = drafts(a, b), took = a.took[b];
    const double u = a.u[b * a.ldu + a.k];
    Row row = row_of(a, b, n, took);
    for (int j = tid; j <= a.k; j += kThreads)
        if (j != took) a.out[b * a.ld_out + j] = j < took ? a.tokens[b * a.ld_tok + j] : -1;
    if (tid == 0) a.accepted[b] = took, found = INT32_MAX, last = -1;

    // the sums' totals, as every wave for itself
    double sr = 0.0, sp = 0.0;
    for (int c = lane; c < a.chunks; c += 64) sr += s[2 * c], sp += s[2 * c + 1];
    int which = 0;
    double total = __shfl(wave_prefix(sr, lane), 63, 64);
    if (!(total > 0.0)) {  // nothing left of p - q: p itself
        total = __shfl(wave_prefix(sp, lane), 63, 64);
        which = 1;
        row.q = nullptr;
        row.drop = -1;
    }
    const double goal = u * total;

    // first chunk whose end is above the goal; without one (u >= 1), the last chunk with anything in it
    int chunk = -1;
    double base = 0.0, run = 0.0;
    for (int c0 = 0; c0 < a.chunks; c0 += 64) {
        const double v = c0 + lane < a.chunks ? s[2 * (c0 + lane) + which] : 0.0;
        const double end = run + wave_prefix(v, lane);
        const uint64_t hit = __ballot(v > 0.0 && end > goal), any = __ballot(v > 0.0);
        if (hit || any) {
            const int l = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(any);
            chunk = c0 + l;
            base = l ? __shfl(end, l - 1, 64) : run;
        }
        if (hit) break;
        run = __shfl(end, 63, 64);
    }
    if (chunk < 0) {  // nothing counts; the same in every wave
        if (tid == 0) a.out[b * a.ld_out + took] = -1;
        return;
    }

    const int64_t lo = (int64_t)chunk * kChunk, hi = lo + kChunk < a.V ? lo + kChunk : a.V;
    const int64_t at = lo + tid * kEach;
    float v[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) v[e] = at + e < hi ? row.r(at + e) : 0.0f;
    double sum = 0.0;
    int32_t end = -1;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        sum += (double)v[e];
        if (v[e] > 0.0f) end = (int32_t)(at + e);
    }
    const double mine = wave_prefix(sum, lane);
    if (lane == 63) part[wave] = mine;
    __syncthreads();
    double before = base;
    for (int w = 0; w < wave; ++w) before += part[w];
    // this thread's entries, one after another
    const double up = __shfl_up(mine, 1, 64);
    double x = lane ? before + up : before;
    int32_t first = -1;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        x += (double)v[e];
        if (v[e] > 0.0f && x > goal && first < 0) first = (int32_t)(at + e);
    }
    const uint64_t hit = __ballot(first >= 0), any = __ballot(end >= 0);
    if (hit && lane == (int)__builtin_ctzll(hit)) atomicMin(&found, first);
    if (any && lane == 63 - (int)__builtin_clzll(any)) atomicMax(&last, end);
    __syncthreads();
    // Rounding may leave the chunk's own last prefix at the goal: its last entry then.
    if (tid == 0) a.out[b * a.ld_out + took] = found < INT32_MAX ? found : last;
}

int chunks_of(int64_t V) { return (int)((V + kChunk - 1) / kChunk); }

}  // namespace

extern "C" size_t pn_spec_workspace(int B, int64_t V)
{
    if (B < 1 || V < 1 || V > INT32_MAX) return 0;
    return (size_t)B * (chunks_of(V) * 2 * sizeof(double) + sizeof(double));
}

extern "C" pn_status pn_spec_verify(const float *target, int64_t ldt, const float *draft, int64_t ldd,
                                    const int32_t *tokens, int64_t ld_tok, const int32_t *n_draft, const float *u,
                                    int64_t ldu, int B, int k, int64_t V, int32_t *out, int64_t ld_out,
                                    int32_t *accepted, void *ws, size_t ws_bytes, void *stream)
{
    if (!target || !u || !out || !accepted || !ws || (!tokens && k > 0)) return PN_EINVAL;
    if (B < 1 || k < 0 || V < 1 || ldt < V || (draft && ldd < V) || ld_tok < k || ldu < (int64_t)k + 1 ||
        ld_out < (int64_t)k + 1)
        return PN_ESHAPE;
    const void *words[] = {target, draft, tokens, n_draft, u, out, accepted};
    for (const void *p : words)
        if (!aligned(p, 4)) return PN_EALIGN;
    if (!aligned(ws, 8)) return PN_EALIGN;
    if (B > 65535 || k > 1024 || V > INT32_MAX) return PN_EUNSUPPORTED;
    if (ws_bytes < pn_spec_workspace(B, V)) return PN_ESHAPE;
    const SpecArgs a = {target, draft, u, tokens, n_draft, out, accepted, (double *)ws,
                        (int32_t *)((double *)ws + (size_t)B * chunks_of(V) * 2), ldt, ldd, ld_tok, ldu, ld_out, V, k,
                        chunks_of(V)};
    const hipStream_t s = (hipStream_t)stream;
    hipLaunchKernelGGL(spec_sums, dim3((unsigned)a.chunks, (unsigned)B), dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    hipLaunchKernelGGL(spec_pick, dim3((unsigned)B), dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    g_last_variant = kVarSpecVerify;
    return PN_OK;
}

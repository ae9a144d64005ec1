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
// workgroup a chunk, and leaves each chunk's sum (and whether p itself has to
// serve, in a second sum); every workgroup finds the row by itself from the
// few gathered probabilities.  Kernel spec_pick, one workgroup a request,
// finds the chunk that holds the border from the sums, then the index within
// it.  A workgroup of one launch never waits for another.
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

// Every wave computes this alike: lane j tests draft j.
__device__ __forceinline__ Row find_row(const SpecArgs &a, int b, int lane)
{
    int n = a.n_draft ? a.n_draft[b] : a.k;
    n = n < 0 ? 0 : n > a.k ? a.k : n;
    int took = n;
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
        if (bad) {
            took = j0 + __builtin_ctzll(bad);
            break;
        }
    }
    Row row;
    row.accepted = took;
    row.p = a.target + ((int64_t)b * (a.k + 1) + took) * a.ldt;
    row.q = took < n && a.draft ? a.draft + ((int64_t)b * a.k + took) * a.ldd : nullptr;
    row.drop = took < n && !a.draft ? a.tokens[b * a.ld_tok + took] : -1;
    return row;
}

// Sum over the workgroup, in every thread.
__device__ __forceinline__ double block_sum(double v, double *part, int lane, int wave)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
    __syncthreads();
    if (lane == 0) part[wave] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kWaves; ++w) v += part[w];
    return v;
}

__global__ __launch_bounds__(kThreads) void spec_sums(SpecArgs a)
{
    __shared__ double part[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.y;
    const Row row = find_row(a, b, lane);
    const int64_t lo = (int64_t)blockIdx.x * kChunk, hi = lo + kChunk < a.V ? lo + kChunk : a.V;
    double sr = 0.0, sp = 0.0;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
        sr += (double)row.r(i);
        sp += (double)clean(row.p[i]);
    }
    sr = block_sum(sr, part, lane, wave);
    sp = block_sum(sp, part, lane, wave);
    if (threadIdx.x == 0) {
        double *s = a.sums + 2 * ((int64_t)b * a.chunks + blockIdx.x);
        s[0] = sr;
        s[1] = sp;
    }
}

// Exclusive prefix of v over the workgroup.
__device__ __forceinline__ double block_before(double v, double *part, int lane, int wave)
{
    double x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 63) part[wave] = x;
    __syncthreads();
    double before = 0.0;
    for (int w = 0; w < wave; ++w) before += part[w];
    const double up = __shfl_up(x, 1, 64);
    return lane == 0 ? before : before + up;
}

__global__ __launch_bounds__(kThreads) void spec_pick(SpecArgs a)
{
    __shared__ double part[kWaves];
    __shared__ int64_t found;
    __shared__ double before_found;
    __shared__ int64_t last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x;
    Row row = find_row(a, b, lane);
    const double *s = a.sums + 2 * (int64_t)b * a.chunks;

    double sr = 0.0, sp = 0.0;
    for (int c = tid; c < a.chunks; c += kThreads) {
        sr += s[2 * c];
        sp += s[2 * c + 1];
    }
    double total = block_sum(sr, part, lane, wave);
    int which = 0;
    if (!(total > 0.0)) {  // nothing left of p - q: p itself
        total = block_sum(sp, part, lane, wave);
        which = 1;
        row.q = nullptr;
        row.drop = -1;
    }
    const double goal = (double)a.u[b * a.ldu + a.k] * total;

    // first chunk whose end is above the goal; without one (u >= 1), the last chunk with anything in it
    if (tid == 0) found = INT64_MAX, last = -1;
    __syncthreads();
    double base = 0.0;
    for (int c0 = 0; c0 < a.chunks; c0 += kThreads) {
        const int c = c0 + tid;
        const double v = c < a.chunks ? s[2 * c + which] : 0.0;
        const double before = base + block_before(v, part, lane, wave);
        const bool hit = v > 0.0 && before + v > goal;
        if (hit) atomicMin((unsigned long long *)&found, (unsigned long long)c);
        if (v > 0.0) atomicMax((long long *)&last, (long long)c);
        __syncthreads();
        if (hit && found == c) before_found = before;
        if (v > 0.0 && found == INT64_MAX && last == c) before_found = before;
        base += block_sum(v, part, lane, wave);
        if (found != INT64_MAX) break;
    }
    __syncthreads();
    const int64_t chunk = found != INT64_MAX ? found : last;
    int32_t token = -1;
    if (chunk >= 0) {  // the same for the whole workgroup
        base = before_found;
        __syncthreads();
        if (tid == 0) found = INT64_MAX, last = -1;
        __syncthreads();
        const int64_t lo = chunk * kChunk, hi = lo + kChunk < a.V ? lo + kChunk : a.V;
        constexpr int kEach = kChunk / kThreads;  // consecutive entries of a thread
        float v[kEach];
        double sum = 0.0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t i = lo + tid * kEach + e;
            v[e] = i < hi ? row.r(i) : 0.0f;
            sum += (double)v[e];
        }
        double run = base + block_before(sum, part, lane, wave);
        int64_t mine = INT64_MAX, end = -1;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            run += (double)v[e];
            const int64_t i = lo + tid * kEach + e;
            if (v[e] > 0.0f) {
                end = i;
                if (run > goal && mine == INT64_MAX) mine = i;
            }
        }
        if (mine != INT64_MAX) atomicMin((unsigned long long *)&found, (unsigned long long)mine);
        if (end >= 0) atomicMax((long long *)&last, (long long)end);
        __syncthreads();
        // Rounding may leave the chunk's own last prefix at the goal: its last entry then.
        token = (int32_t)(found != INT64_MAX ? found : last);
    }
    for (int j = tid; j <= a.k; j += kThreads)
        a.out[b * a.ld_out + j] = j < row.accepted ? a.tokens[b * a.ld_tok + j] : j == row.accepted ? token : -1;
    if (tid == 0) a.accepted[b] = row.accepted;
}

int chunks_of(int64_t V) { return (int)((V + kChunk - 1) / kChunk); }

}  // namespace

extern "C" size_t pn_spec_workspace(int B, int64_t V)
{
    if (B < 1 || V < 1 || V > INT32_MAX) return 0;
    return (size_t)B * chunks_of(V) * 2 * sizeof(double);
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
    const SpecArgs a = {target, draft, u, tokens, n_draft, out, accepted, (double *)ws, ldt, ldd, ld_tok, ldu, ld_out,
                        V, k, chunks_of(V)};
    const hipStream_t s = (hipStream_t)stream;
    hipLaunchKernelGGL(spec_sums, dim3((unsigned)a.chunks, (unsigned)B), dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    hipLaunchKernelGGL(spec_pick, dim3((unsigned)B), dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return PN_ELAUNCH;
    g_last_variant = kVarSpecVerify;
    return PN_OK;
}

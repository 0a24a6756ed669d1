// logprobs.cu -- log probabilities of given tokens, their ranks, the entropy and
// the most probable alternatives, from logits read once.
//
//   m = max x, l = sum e^(x - m), s = sum (x - m) e^(x - m)
//   log p(t) = x_t - m - log l,  H = log l - s / l,  rank = #{i: x_i > x_t}
//
// A row goes to a cluster of 1 to 8 CTAs, each of which takes a part of it in
// chunks of 16 values a thread, the next chunk's loads under way while it works on
// one. A thread keeps its own m, l and s (FP32, a few hundred terms each) and
// rescales them when its maximum grows; they are joined at the end, over lanes,
// warps and the cluster's CTAs.
//
// Alternatives: a value and its index make a 64-bit key, larger for the larger
// value and, among equal ones, for the lower index, so that no two are equal. Values
// above a bound that at least k values reach are collected in shared memory. The
// first bound is the k-th largest of the maxima of 32 groups of a chunk; when a chunk
// leaves kMany candidates or more, they are ranked by counting (a key's rank is the
// number of larger ones), the first k kept, and the k-th is the new bound. Later
// values equal to the bound lose to those that are there by their index.
#include "common.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 16;                     // values of a chunk a thread
constexpr int kChunk = kThreads * kPer;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kMany = 128;                   // candidates that are ranked at once
constexpr int kBatch = 1024;                 // keys ranked together, two a thread
constexpr int kCap = kChunk + kMany;
constexpr float kLog2e = 1.4426950408889634f;

struct LogprobParams {
    const void* x;
    int64_t stride;
    const void* tok;
    int tok_type;
    int V, k;
    float* lp;
    int* ranks;
    float* entropy;
    int* top_ids;
    float* top_lp;
};

struct Stats {
    float m, l, s;
    int above;
};

struct TopSmem {
    alignas(16) uint64_t best[kMaxTop];      // in order
    alignas(16) uint64_t work[kBatch];
    alignas(16) uint64_t cand[kCap];
};

struct Smem {
    Stats part[kWarps];
    Stats all;                               // this CTA's, read by the cluster's first
    float group[2 * kWarps];
    int count;
};

// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Ordered as the floats are (-0 below 0 like its bits: made one by the caller).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u ^ (u & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u)
{
    return __uint_as_float(u ^ (u & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i)
{
    return static_cast<uint64_t>(ordered(x + 0.0f)) << 32 | (0xFFFFFFFFu - i);
}

// Statistics over m = max(a.m, b.m); an empty side (m -inf) changes nothing.
__device__ __forceinline__ Stats join(const Stats& a, const Stats& b)
{
    Stats r;
    r.m = max_nan(a.m, b.m);
    r.above = a.above + b.above;
    r.l = r.s = 0.0f;
    if (a.m != -INFINITY) {
        const float d = a.m - r.m, f = ex2(d * kLog2e);
        r.l += a.l * f;
        r.s += f == 0.0f ? 0.0f : (a.s + d * a.l) * f;
    }
    if (b.m != -INFINITY) {
        const float d = b.m - r.m, f = ex2(d * kLog2e);
        r.l += b.l * f;
        r.s += f == 0.0f ? 0.0f : (b.s + d * b.l) * f;
    }
    return r;
}

__device__ __forceinline__ Stats warp_join(Stats a)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stats b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
        b.l = __shfl_xor_sync(0xffffffffu, a.l, o);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
        b.above = __shfl_xor_sync(0xffffffffu, a.above, o);
        a = join(a, b);
    }
    return a;
}

// The first k of n candidates to t.best in order (fewer if there are fewer); all
// threads. Returns how many.
__device__ __noinline__ int rank_candidates(TopSmem& t, int n, int k)
{
    const int tid = threadIdx.x;
    int kept = 0;
    for (int pos = 0; pos < n;) {
        // the kept ones and as many others as make a batch
        const int take = min(n - pos, kBatch - kept), m = kept + take, even = (m + 1) & ~1;
        for (int i = tid; i < even; i += kThreads)
            t.work[i] = i < kept ? t.best[i] : (i < m ? t.cand[pos + i - kept] : 0ull);
        __syncthreads();
        uint64_t mine[2];
        int rank[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) mine[i] = tid + i * kThreads < m ? t.work[tid + i * kThreads] : 0ull;
        const ulonglong2* all = reinterpret_cast<const ulonglong2*>(t.work);
        if (tid < m) {
#pragma unroll 4
            for (int i = 0; i < even / 2; ++i) {
                const ulonglong2 x = all[i];
                rank[0] += (x.x > mine[0]) + (x.y > mine[0]);
                rank[1] += (x.x > mine[1]) + (x.y > mine[1]);
            }
        }
        // (best is read no more)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (tid + i * kThreads < m && rank[i] < k) t.best[rank[i]] = mine[i];
        kept = min(m, k);
        pos += take;
        __syncthreads();
    }
    return kept;
}

template <typename T>
struct Raw;
template <>
struct Raw<float> {
    static constexpr int kVec = 4;
    float4 r;
    __device__ void load(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
    __device__ void put(int i, float x) { (&r.x)[i] = x; }
    __device__ float get(int i) const { return (&r.x)[i]; }
};
template <>
struct Raw<__nv_bfloat16> {
    static constexpr int kVec = 8;
    uint4 r;
    __device__ void load(const __nv_bfloat16* p) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ void put(int i, __nv_bfloat16 x)
    {
        uint32_t& w = (&r.x)[i >> 1];
        const uint32_t u = *reinterpret_cast<const uint16_t*>(&x);
        w = i & 1 ? (w & 0xFFFFu) | u << 16 : (w & 0xFFFF0000u) | u;
    }
    __device__ float get(int i) const
    {
        const uint32_t w = (&r.x)[i >> 1];
        return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    }
};
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float lowest(float) { return -INFINITY; }
__device__ __forceinline__ __nv_bfloat16 lowest(__nv_bfloat16) { return __ushort_as_bfloat16(0xFF80); }

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 2) token_logprobs_kernel(const LogprobParams p)
{
    constexpr int VEC = Raw<T>::kVec, NV = kPer / VEC;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    TopSmem& top = *reinterpret_cast<TopSmem*>(smem_raw);
    __shared__ Smem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int64_t row = blockIdx.x / ctas;
    const T* const x = static_cast<const T*>(p.x) + row * p.stride;
    // 16-byte pieces of memory: piece j has values VEC j - shift .. + VEC - 1
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const uint32_t pieces = (static_cast<uint32_t>(p.V) + shift + VEC - 1) / VEC;
    // this CTA's pieces: whole chunks but for the last CTA's
    const uint32_t chunks = (pieces + kThreads * NV - 1) / (kThreads * NV);
    const uint32_t c0 = static_cast<uint64_t>(chunks) * rank / ctas, c1 = static_cast<uint64_t>(chunks) * (rank + 1) / ctas;
    const int64_t tok = load_slot(p.tok, p.tok_type, row);
    const bool given = tok >= 0 && tok < p.V;
    const float xt = given ? as_float(x[tok]) : INFINITY;

    auto first_of = [&](uint32_t c, int v) { return static_cast<int64_t>(c * NV + v) * (kThreads * VEC) + tid * VEC - shift; };
    Raw<T> next[NV];
    auto load = [&](uint32_t c) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t i = first_of(c, v);
            if (i >= 0 && i + VEC <= p.V) {
                next[v].load(x + i);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) next[v].put(e, i + e >= 0 && i + e < p.V ? x[i + e] : lowest(T()));
            }
        }
    };
    if (TOP && tid == 0) sm.count = 0;
    Stats st = {-INFINITY, 0.0f, 0.0f, 0};
    float bound = -INFINITY;
    bool full = false;                       // k values that reach the bound are there
    int n = 0;                               // candidates
    if (c0 < c1) load(c0);
#pragma unroll 1
    for (uint32_t c = c0; c < c1; ++c) {
        float v[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = next[e / VEC].get(e % VEC);
        if (c + 1 < c1) load(c + 1);
        float mx = v[0];
#pragma unroll
        for (int e = 1; e < kPer; ++e) mx = max_nan(mx, v[e]);
        // ---- the running statistics ----
        const float m = max_nan(st.m, mx);
        if (m != st.m) {
            if (st.m != -INFINITY) {
                const float d = st.m - m, f = ex2(d * kLog2e);
                st.s = f == 0.0f ? 0.0f : (st.s + d * st.l) * f;
                st.l *= f;
            }
            st.m = m;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            // (a value of -inf, whose product with its weight of 0 would be NaN: -2^100)
            const float d = max_nan(v[e] - ref, -0x1p100f);
            const float w = ex2(d * kLog2e);
            st.l += w;
            st.s += d * w;
            st.above += v[e] > xt;
        }
        if (!TOP) continue;
        // ---- candidates ----
        const bool was_full = full;
        if (!full) {
            float g = mx;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
            if ((lane & 15) == 0) sm.group[tid >> 4] = g;
            __syncthreads();
            g = sm.group[lane];
            int higher = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float o = __shfl_sync(0xffffffffu, g, i);
                higher += o > g || (o == g && i < lane);
            }
            bound = __shfl_sync(0xffffffffu, g, __ffs(__ballot_sync(0xffffffffu, higher == p.k - 1)) - 1);
            full = bound > -INFINITY;
        }
        if (was_full ? mx > bound : mx >= bound) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int64_t i = first_of(c, e / VEC) + e % VEC;
                if ((was_full ? v[e] > bound : v[e] >= bound) && i >= 0 && i < p.V)
                    top.cand[atomicAdd(&sm.count, 1)] = key_of(v[e], static_cast<uint32_t>(i));
            }
        }
        __syncthreads();
        n = sm.count;
        if (n >= kMany) {
            const int kept = rank_candidates(top, n, p.k);
            // (the kept ones are candidates again)
            if (tid < kept) top.cand[tid] = top.best[tid];
            if (tid == 0) sm.count = kept;
            if (kept == p.k) {
                bound = unordered(static_cast<uint32_t>(top.best[p.k - 1] >> 32));
                full = true;
            }
            n = kept;
        }
        __syncthreads();
    }
    // ---- this CTA's statistics and alternatives ----
    st = warp_join(st);
    if (lane == 0) sm.part[warp] = st;
    __syncthreads();
    if (warp == 0) {
        st = sm.part[lane & (kWarps - 1)];
        if (lane >= kWarps) st = {-INFINITY, 0.0f, 0.0f, 0};
        st = warp_join(st);
        if (lane == 0) sm.all = st;
    }
    if (TOP) {
        const int kept = rank_candidates(top, n, p.k);
        if (tid == 0) sm.count = kept;
    }
    if (ctas > 1) cluster.sync();
    else __syncthreads();
    if (rank == 0) {
        if (ctas > 1) {
            if (warp == 0) {
                st = {-INFINITY, 0.0f, 0.0f, 0};
                if (lane < ctas) st = *cluster.map_shared_rank(&sm.all, lane);
                st = warp_join(st);
                if (lane == 0) sm.part[0] = st;
            }
            if (TOP) {
                // lists one behind another; empty places are zeros, the lowest key
                for (int i = tid; i < static_cast<int>(ctas) * p.k; i += kThreads) {
                    const int r = i / p.k, j = i - r * p.k;
                    const TopSmem* far = cluster.map_shared_rank(&top, r);
                    top.cand[i] = j < *cluster.map_shared_rank(&sm.count, r) ? far->best[j] : 0ull;
                }
            }
        } else if (tid == 0) {
            sm.part[0] = sm.all;
        }
        __syncthreads();
        if (TOP && ctas > 1) rank_candidates(top, ctas * p.k, p.k);
        const Stats all = sm.part[0];
        // nothing but -inf: no distribution, the sum is 0. A NaN or +inf: the sum is NaN.
        const float logl = logf(all.l);
        const bool bad = !(all.l >= 0.0f);
        auto logp = [&](float v) { return v == -INFINITY && !bad ? -INFINITY : v - all.m - logl; };
        if (tid == 0) {
            p.lp[row] = given ? logp(xt) : NAN;
            if (p.ranks) p.ranks[row] = given && !bad ? all.above : -1;
            if (p.entropy) p.entropy[row] = all.l == 0.0f ? 0.0f : logl - all.s / all.l;
        }
        if (TOP && tid < p.k) {
            const uint64_t key = top.best[tid];
            p.top_ids[row * p.k + tid] = bad ? -1 : static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
            p.top_lp[row * p.k + tid] = bad ? NAN : logp(unordered(static_cast<uint32_t>(key >> 32)));
        }
    }
    // (the others' shared memory is read until here)
    if (ctas > 1) cluster.sync();
}

template <typename T, bool TOP>
cudaError_t launch(const LogprobParams& p, int64_t R, int ctas, cudaStream_t st)
{
    const size_t smem = TOP ? sizeof(TopSmem) : 0;
    if (TOP) {
        const cudaError_t e = cudaFuncSetAttribute(token_logprobs_kernel<T, TOP>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(R * ctas));
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, token_logprobs_kernel<T, TOP>, p);
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_token_logprobs(const void* logits, int dtype, int64_t row_stride, const void* tokens,
                                       int token_type, int64_t num_rows, int V, float* logprobs, int32_t* ranks,
                                       float* entropy, int top, int32_t* top_ids, float* top_logprobs, void* stream)
{
    const char* name = "pa_token_logprobs";
    PA_REQUIRE(num_rows == 0 || (logits && tokens && logprobs), PA_ERR_NULLPTR, "%s: NULL tensor pointer", name);
    PA_REQUIRE(num_rows >= 0 && V > 0 && top >= 0, PA_ERR_INVALID, "%s: empty or negative size", name);
    PA_REQUIRE(dtype == PA_DTYPE_F32 || dtype == PA_DTYPE_BF16, PA_ERR_INVALID, "%s: unknown dtype %d", name, dtype);
    PA_REQUIRE(token_type == PA_INDEX_I32 || token_type == PA_INDEX_I64, PA_ERR_INVALID, "%s: unknown token type %d",
               name, token_type);
    PA_REQUIRE(top <= V, PA_ERR_INVALID, "%s: %d alternatives of %d tokens", name, top, V);
    PA_REQUIRE(top <= kMaxTop, PA_ERR_UNSUPPORTED, "%s: %d alternatives (at most %d)", name, top, kMaxTop);
    PA_REQUIRE(top == 0 || num_rows == 0 || (top_ids && top_logprobs), PA_ERR_NULLPTR,
               "%s: NULL top_ids or top_logprobs", name);
    PA_REQUIRE(num_rows <= 1 || row_stride >= V, PA_ERR_INVALID, "%s: rows overlap (row_stride below V)", name);
    PA_REQUIRE(V <= 0x7FFFFFFF - 2 * kChunk && num_rows <= 0x7FFFFFFF / kMaxCluster, PA_ERR_UNSUPPORTED,
               "%s: too many rows or tokens", name);
    PA_REQUIRE(aligned(logits, dtype == PA_DTYPE_F32 ? 4 : 2) && aligned(tokens, token_type == PA_INDEX_I64 ? 8 : 4) &&
                   aligned(logprobs, 4) && aligned(ranks, 4) && aligned(entropy, 4) && aligned(top_ids, 4) &&
                   aligned(top_logprobs, 4),
               PA_ERR_INVALID, "%s: misaligned pointer", name);
    if (num_rows == 0) return PA_OK;
    const int sms = device_sm_count();
    PA_REQUIRE(sms > 0, PA_ERR_CUDA, "%s: cannot query the device", name);
    LogprobParams p;
    p.x = logits;
    p.stride = num_rows > 1 ? row_stride : 0;
    p.tok = tokens;
    p.tok_type = token_type;
    p.V = V;
    p.k = top;
    p.lp = logprobs;
    p.ranks = ranks;
    p.entropy = entropy;
    p.top_ids = top_ids;
    p.top_lp = top_logprobs;
    // As many CTAs a row as fill the GPU, two an SM, and have a chunk each.
    int ctas = kMaxCluster;
    while (ctas > 1 && (num_rows * (ctas / 2) >= 2 * sms || V <= kChunk * (ctas / 2))) ctas /= 2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == PA_DTYPE_F32) e = top ? launch<float, true>(p, num_rows, ctas, st) : launch<float, false>(p, num_rows, ctas, st);
    else e = top ? launch<__nv_bfloat16, true>(p, num_rows, ctas, st) : launch<__nv_bfloat16, false>(p, num_rows, ctas, st);
    PA_REQUIRE(e == cudaSuccess, PA_ERR_CUDA, "%s: launch: %s", name, cudaGetErrorString(e));
    return check_launch(name);
}

// logprobs.cu -- log probabilities of given tokens, their ranks, the entropy and
// the most probable alternatives, from logits read once.
//
//   m = max x, l = sum e^(x - m), s = sum (x - m) e^(x - m)
//   log p(t) = x_t - m - log l,  H = log l - s / l,  rank = #{i: x_i > x_t}
//
// A row goes to a cluster of 1 to 8 CTAs, each of which takes a part of it in chunks
// of 64 bytes a thread, and a cluster takes one row after another. A thread copies its
// own pieces of the next three chunks, the next row's among them, to shared memory (so
// that no barrier stands between a copy and its use), keeps its own m, l and s (FP32, a
// few hundred terms each) and rescales them when a value passes m by more than kRaise (m
// need not be the maximum, and in the first chunks some lane's grows nearly every time);
// they are joined at a row's end, over lanes, warps and the cluster's CTAs. A value's
// exponent is one fused operation, x log2 e - c with c = m log2 e as rounded; what the
// rounding is off by is one factor of all terms since m last grew, taken out of their sums.
// (Past 2^10 that factor is no longer near 1: there, and where a term is -inf, x - m is
// formed first.) The rank counts signs of x_t - x, or pairs of BF16 ones, only where a
// thread's 16 values have a larger one: a comparison and a sum for each took 250 rows x
// 131072 from 24.8 to 28.9 us.
//
// Alternatives: a value and its index make a 64-bit key, larger for the larger
// value and, among equal ones, for the lower index, so that no two are equal. The pass
// itself does nothing for them, a thread's maximum is there anyhow. Behind it the k-th
// largest of the maxima of 32 groups of threads is a bound that k values at least
// reach; the threads whose maximum does, k to twice as many, have their pieces read
// again (from L2, a piece a lane), and values that reach the bound go to a list in
// shared memory, which is put in order by counting (a key's rank is the number of larger
// ones): by one warp without a barrier if there are at most 64, else by all, and more
// than kShort are thinned first, by the same bound over 32 groups of the list; one that
// runs over (thousands of equal values) is made anew by `careful`, which keeps it short as
// it goes. -inf is never listed: where fewer than k values are finite the lowest indices
// of the others follow.
//
// What bounds it: many long rows without alternatives, the reads (4096 rows x 50000 FP32 129
// us, 6.4 TB/s; a copy's rate would take 121). A row a CTA, what stands around the reads: the two
// loads of the token's logit, one behind the other, 2 us, and 5 us of joins, bound, second
// reading and order, every instruction of which runs once and out of a cold cache (250 rows
// x 131072 BF16 with 20 alternatives 25 us, without 20.5; 38 such rows 14.4; one row of 32003
// FP32 with 5 alternatives 8.2, 6.5 in a graph). A CTA's rows have these ends one behind
// another: 4096 x 50000 FP32 with 20 alternatives 206 us, 4096 x 13000 BF16 59 without and 92
// with them, where the reads are 16. A -inf among a thread's 16 values has their exponentials
// formed twice: 250 x 131072 BF16 of which 1% or 99% are masked 33 us. All four forms are held
// to 64 registers for two CTAs an SM and spill 4 to 36 bytes. Rows cut over clusters at
// any number of rows cost more in joins than they balance (250 rows on 2, 4 and 8 CTAs 37, 60,
// 108 us, when one took 29).
#include "common.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPieces = 4;                   // 16-byte pieces of a chunk a thread
constexpr int kStages = 3;                   // chunks on their way
constexpr uint32_t kSlot = kPieces * kThreads * 16;   // bytes of a chunk
constexpr int kPer = 16;                     // values a thread has in registers at once
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kList = 1024;                  // candidates
constexpr int kShort = 256;                  // of which at most so many are put in order
constexpr float kRaise = 8.0f;               // what values may pass the thread's m by
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast = -0x1.fffffep127f;

struct LogprobParams {
    const void* x;
    int64_t stride;
    const void* tok;
    int tok_type;
    int64_t R;
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
    alignas(16) uint64_t work[kShort + 8];
    alignas(16) uint64_t list[kList];
    alignas(16) uint64_t far[kMaxCluster * kMaxTop + 8];   // the first's: every CTA's best
};

struct Smem {
    Stats part[2][kWarps];                   // by row parity
    Stats all[kMaxCluster];                  // the first's: every CTA's
    float group[2 * kWarps];
    uint16_t who[kThreads];                  // threads whose maximum reaches the bound
    int threads[2], count[2];                // by row parity
    float bound;
    int left;
};

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

// The lanes' statistics over their common maximum. (An empty lane's m is -inf and adds
// nothing; a NaN is in the sums, not in m, and stays there.)
__device__ __forceinline__ Stats warp_join(Stats a)
{
    const float m = warp_max_f32(a.m), d = a.m - m;
    const float f = a.m == m ? 1.0f : ex2(d * kLog2e);
    a.s = f == 1.0f ? a.s : (f == 0.0f ? 0.0f : (a.s + d * a.l) * f);
    a.l *= f;
    a.m = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.l += __shfl_xor_sync(0xffffffffu, a.l, o);
        a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    }
    a.above = __reduce_add_sync(0xffffffffu, a.above);
    return a;
}

// A value that the k-th largest (k <= 32) of the lanes' reaches, the same but for the
// lower half of its bits: bit by bit, how many lanes have what is fixed and a one.
__device__ __forceinline__ uint32_t kth_of_lanes(uint32_t x, int k)
{
    bool in = true;
    uint32_t bits = 0;
#pragma unroll
    for (int b = 31; b >= 16; --b) {
        const uint32_t ones = __ballot_sync(0xffffffffu, in && (x >> b & 1));
        const bool one = __popc(ones) >= k;
        if (one) bits |= 1u << b;
        else k -= __popc(ones);
        in = in && (x >> b & 1) == one;
    }
    return bits;
}

// The first k of the n <= kShort keys at `keys` (16-byte aligned, room for eight more)
// to `best` in order; all threads, a barrier before and after.
__device__ __forceinline__ void put_in_order(uint64_t* best, uint64_t* keys, int n, int k)
{
    const int tid = threadIdx.x, end = (n + 7) & ~7;
    if (tid >= n && tid < end) keys[tid] = 0;             // (below every key)
    __syncthreads();
    if (tid < n) {
        const uint64_t mine = keys[tid];
        const ulonglong2* all = reinterpret_cast<const ulonglong2*>(keys);
        int rank = 0;
#pragma unroll 1
        for (int i = 0; i < end / 2; i += 4) {
            ulonglong2 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = all[i + j];
#pragma unroll
            for (int j = 0; j < 4; ++j) rank += (x[j].x > mine) + (x[j].y > mine);
        }
        if (rank < k) best[rank] = mine;
    }
    __syncthreads();
}

// The first k of the list's n keys to t.best in order (fewer if there are fewer); all
// threads, a barrier before and after. A long list is taken kShort at a time, the first
// k of what was there among them, after what no group of 32 needs has left it.
__device__ __noinline__ int first_of_list(TopSmem& t, Smem& sm, int n, int k)
{
    const int tid = threadIdx.x, lane = tid & 31;
    if (n > kShort) {
        // values that the k-th largest of 32 groups' maxima reach, in place: a thread
        // holds its keys while the others take theirs
        uint64_t key[kList / kThreads];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kList / kThreads; ++i) {
            key[i] = tid + i * kThreads < n ? t.list[tid + i * kThreads] : 0ull;
            m = max(m, static_cast<uint32_t>(key[i] >> 32));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((lane & 15) == 0) sm.group[tid >> 4] = __uint_as_float(m);
        if (tid == 0) sm.left = 0;
        __syncthreads();
        const uint32_t bound = kth_of_lanes(__float_as_uint(sm.group[lane]), k);
#pragma unroll
        for (int i = 0; i < kList / kThreads; ++i)
            if (tid + i * kThreads < n && static_cast<uint32_t>(key[i] >> 32) >= bound)
                t.list[atomicAdd(&sm.left, 1)] = key[i];
        __syncthreads();
        n = sm.left;
    }
    int kept = 0;
    for (int pos = 0; pos < n;) {
        const int take = min(n - pos, kShort - kept);
        if (tid < kept + take) t.work[tid] = tid < kept ? t.best[tid] : t.list[pos + tid - kept];
        put_in_order(t.best, t.work, kept + take, k);
        kept = min(kept + take, k);
        pos += take;
    }
    return kept;
}

// The same for n <= 64 keys, by the first warp alone: no barrier.
__device__ __forceinline__ int first_of_few(TopSmem& t, int n, int k, int lane)
{
    if (lane == 0) t.list[n] = 0;
    __syncwarp();
    const uint64_t a = lane < n ? t.list[lane] : 0ull, b = lane + 32 < n ? t.list[lane + 32] : 0ull;
    int ra = 0, rb = 0;
#pragma unroll 4
    for (int i = 0; i < n; i += 2) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(t.list + i);
        ra += (x.x > a) + (x.y > a);
        rb += (x.x > b) + (x.y > b);
    }
    if (lane < n && ra < k) t.best[ra] = a;
    if (lane + 32 < n && rb < k) t.best[rb] = b;
    __syncwarp();
    return min(n, k);
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float lowest(float) { return -INFINITY; }
__device__ __forceinline__ __nv_bfloat16 lowest(__nv_bfloat16) { return __ushort_as_bfloat16(0xFF80); }

__device__ __forceinline__ void unpack(const uint4& r, float* v, float)
{
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const uint4& r, float* v, __nv_bfloat16)
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// A CTA's part of a row: 16-byte pieces of memory, piece j with the values VEC j - shift
// .. + VEC - 1, in chunks [c0, c1) of kPieces pieces a thread.
template <typename T>
struct Part {
    static constexpr int VEC = 16 / sizeof(T);
    const T* x;
    int V, shift;
    uint32_t c0, c1;

    __device__ __forceinline__ Part(const LogprobParams& p, int64_t row, uint32_t rank, uint32_t ctas)
    {
        x = static_cast<const T*>(p.x) + row * p.stride;
        V = p.V;
        shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
        const uint32_t pieces = (static_cast<uint32_t>(V) + shift + VEC - 1) / VEC;
        const uint32_t chunks = (pieces + kThreads * kPieces - 1) / (kThreads * kPieces);
        c0 = chunks * rank / ctas;
        c1 = chunks * (rank + 1) / ctas;
    }
    // the first value of this thread's first piece of a chunk; the next pieces are
    // kThreads VEC values further
    __device__ __forceinline__ int first_of(uint32_t c) const
    {
        return static_cast<int>(c * (kThreads * kPieces * VEC) + threadIdx.x * VEC) - shift;
    }
    // This thread's pieces of the chunk whose first value for it is i0, on their way to
    // shared memory at dst, dst + 16 kThreads, ..
    __device__ __forceinline__ void fetch(int i0, uint32_t dst) const
    {
        constexpr int kSpan = (kPieces - 1) * kThreads * VEC + VEC;
        if (V >= kSpan && static_cast<uint32_t>(i0) <= static_cast<uint32_t>(V - kSpan)) {
            const T* const at = x + i0;
#pragma unroll
            for (int v = 0; v < kPieces; ++v)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + v * (16 * kThreads)),
                             "l"(at + v * (kThreads * VEC))
                             : "memory");
            return;
        }
#pragma unroll 1
        for (int v = 0; v < kPieces; ++v) {
            const int i = i0 + v * (kThreads * VEC);
            T* const at = static_cast<T*>(__cvta_shared_to_generic(dst + v * (16 * kThreads)));
            if (i >= 0 && i + VEC <= V) {
                cp_async16(at, x + i, 16);
            } else {
                for (int e = 0; e < VEC; ++e) at[e] = i + e >= 0 && i + e < V ? x[i + e] : lowest(T());
            }
        }
    }
};

// The candidates of a part whose list ran over: the first k of those behind are kept, a
// value a thread at a time. Returns the list's length.
template <typename T>
__device__ __noinline__ int careful(TopSmem& t, Smem& sm, int& count, const T* x, int begin, int end, int k)
{
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) count = 0;
    __syncthreads();
    float bound = -INFINITY;
    static_assert(kShort + kThreads <= kList, "the list has room for what is kept and a value a thread");
    for (int at = begin; at < end; at += kThreads) {
        const int i = at + tid;
        const float v = i < end ? as_float(x[i]) : -INFINITY;
        // (what equals the bound comes behind those that are there)
        if (v > bound) t.list[atomicAdd(&count, 1)] = key_of(v, static_cast<uint32_t>(i));
        __syncthreads();
        const int n = count;
        if (n >= kShort) {
            const int kept = first_of_list(t, sm, n, k);
            if (tid < kept) t.list[tid] = t.best[tid];
            if (tid == 0) count = kept;
            if (kept == k) bound = unordered(static_cast<uint32_t>(t.best[k - 1] >> 32));
        }
        __syncthreads();
    }
    return count;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 2) token_logprobs_kernel(const LogprobParams p)
{
    constexpr int VEC = Part<T>::VEC;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint4* const ring = reinterpret_cast<uint4*>(smem_raw) + threadIdx.x;
    TopSmem& top = *reinterpret_cast<TopSmem*>(smem_raw + kStages * kSlot);
    __shared__ Smem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int64_t step = gridDim.x / ctas;
    if (ctas > 1) cluster.barrier_arrive();
    if (TOP && tid == 0) sm.count[0] = sm.threads[0] = 0; // (ahead of the first row's barriers)

    auto token = [&](int64_t row) { return row < p.R ? load_slot(p.tok, p.tok_type, row) : -1; };
    auto logit = [&](int64_t row, int64_t t) {
        return t >= 0 && t < p.V ? as_float(static_cast<const T*>(p.x)[row * p.stride + t]) + 0.0f : INFINITY;   // (-0 as 0)
    };
    int64_t tok = token(blockIdx.x / ctas);

    // ---- the next chunks on their way, over the row's end ----
    int64_t a_row = blockIdx.x / ctas;
    Part<T> a_part(p, a_row, rank, ctas);
    uint32_t a_left = a_part.c1 - a_part.c0;
    int a_i0 = a_part.first_of(a_part.c0);
    const uint32_t ring_at = smem_u32(ring);
    uint32_t a_slot = 0, slot = 0;
    auto fetch = [&] {
        while (a_left == 0 && a_row < p.R) {
            a_row += step;
            if (a_row >= p.R) break;
            a_part = Part<T>(p, a_row, rank, ctas);
            a_left = a_part.c1 - a_part.c0;
            a_i0 = a_part.first_of(a_part.c0);
        }
        if (a_left > 0) {
            a_part.fetch(a_i0, ring_at + a_slot);
            a_i0 += kThreads * kPieces * VEC;
            --a_left;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        a_slot = a_slot + kSlot == kStages * kSlot ? 0 : a_slot + kSlot;
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch();
    float xt = logit(blockIdx.x / ctas, tok);
    int parity = 0;
#pragma unroll 1
    for (int64_t row = blockIdx.x / ctas; row < p.R; row += step, parity ^= 1) {
        const Part<T> part(p, row, rank, ctas);
        const int64_t tok_next = token(row + step);
        Stats st = {-INFINITY, 0.0f, 0.0f, 0};            // (s in units of log2)
        float c_now = 0.0f, off = 0.0f;                  // c, and c - m log2 e
        float most = -INFINITY, raise_at = -INFINITY;    // the thread's maximum; m + kRaise
        float l_raw = 0.0f, s_raw = 0.0f;                // sums over c since m last grew
        auto settle = [&] {
            st.l += fmaf(l_raw, off * kLn2, l_raw);
            st.s += fmaf(off, fmaf(s_raw, kLn2, l_raw), s_raw);
            l_raw = s_raw = 0.0f;
        };
#pragma unroll 1
        for (uint32_t c = part.c0; c < part.c1; ++c) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            const uint4* const in = ring + slot / 16;
#pragma unroll 1
            for (int at = 0; at < kPieces; at += kPer / VEC) {
                float w[kPer];
#pragma unroll
                for (int i = 0; i < kPer / VEC; ++i) unpack(in[(at + i) * kThreads], w + i * VEC, T());
                float mx = w[0];
#pragma unroll
                for (int e = 1; e < kPer; e += 2) mx = max3(mx, w[e], w[e + 1 < kPer ? e + 1 : e]);
                // the token's rank (of a probable one few threads have values above it)
                if (mx > xt) {
                    if constexpr (VEC == 4) {
                        // signs of xt - x
                        uint32_t signs = 0;
#pragma unroll
                        for (int e = 0; e < kPer; e += 2) {
                            const float2 d = __ffma2_rn(make_float2(w[e], w[e + 1]), make_float2(-1.f, -1.f), make_float2(xt, xt));
                            signs = __funnelshift_l(__float_as_uint(d.x), signs, 1);
                            signs = __funnelshift_l(__float_as_uint(d.y), signs, 1);
                        }
                        st.above += __popc(signs);
                    } else {
                        // ones, pair by pair (8 at most, BF16 exactly)
                        const __nv_bfloat162 t2 = __float2bfloat162_rn(xt);
                        __nv_bfloat162 n2 = __float2bfloat162_rn(0.0f);
#pragma unroll
                        for (int i = 0; i < kPer / VEC; ++i) {
                            const uint4 r = in[(at + i) * kThreads];
                            n2 = __hadd2(n2, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&r.x), t2));
                            n2 = __hadd2(n2, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&r.y), t2));
                            n2 = __hadd2(n2, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&r.z), t2));
                            n2 = __hadd2(n2, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&r.w), t2));
                        }
                        st.above += static_cast<int>(__low2float(n2) + __high2float(n2));
                    }
                }
                most = fmaxf(most, mx);
                if (mx > raise_at) {
                    settle();
                    if (st.m != -INFINITY) {
                        const float d = (st.m - mx) * kLog2e, f = ex2(d);
                        st.s = f == 0.0f ? 0.0f : (st.s + d * st.l) * f;
                        st.l *= f;
                    }
                    st.m = mx;
                    raise_at = mx + kRaise;
                    c_now = mx * kLog2e;
                    off = fabsf(mx) <= 1024.0f ? fmaf(-mx, kLog2e, c_now) : 0.0f;
                }
                float dot = NAN;
                float2 l = make_float2(0.f, 0.f);
                if (fabsf(st.m) <= 1024.0f) {
                    const float2 neg = make_float2(-c_now, -c_now), log2e = make_float2(kLog2e, kLog2e);
                    float2 s = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < kPer; e += 2) {
                        const float2 y = __ffma2_rn(make_float2(w[e], w[e + 1]), log2e, neg);
                        const float2 x = make_float2(ex2(y.x), ex2(y.y));
                        l = __fadd2_rn(l, x);
                        s = __ffma2_rn(y, x, s);
                    }
                    dot = s.x + s.y;
                }
                if (dot == dot) {
                    l_raw += l.x + l.y;
                    s_raw += dot;
                } else {
                    // past the range, or -inf among them, whose product with its weight
                    // of 0 is NaN. (One among the values makes both sums NaN.)
                    const float ref = st.m == -INFINITY ? 0.0f : st.m;
                    float sum = 0.0f;
                    dot = 0.0f;
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        const float y = (w[e] - ref) * kLog2e, x = ex2(y);
                        sum += x;
                        dot += x == 0.0f ? 0.0f : y * x;
                    }
                    st.l += sum;
                    st.s += dot;
                }
            }
            slot = slot + kSlot == kStages * kSlot ? 0 : slot + kSlot;
            fetch();                         // (into the slot just read: this thread's own)
        }
        settle();
        st.s *= kLn2;
        const float xt_next = logit(row + step, tok_next);
        // ---- this CTA's statistics and alternatives, to the cluster's first ----
        const float mine = most;
        st = warp_join(st);
        if (lane == 0) sm.part[parity][warp] = st;
        if (TOP) {
            float g = mine;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
            if ((lane & 15) == 0) sm.group[tid >> 4] = g;
        }
        __syncthreads();
        if (warp == 0) {
            st = sm.part[parity][lane & (kWarps - 1)];
            if (lane >= kWarps) st = {-INFINITY, 0.0f, 0.0f, 0};
            st = warp_join(st);
        }
        int kept = 0;
        if (TOP) {
            // (a group of -inf counts as one of the least finite value)
            if (warp == 0) {
                const uint32_t low = kth_of_lanes(ordered(fmaxf(sm.group[lane], kLeast)), p.k);
                if (lane == 0) sm.bound = unordered(max(low, ordered(kLeast)));
            }
            __syncthreads();
            const float bound = sm.bound;
            int &threads = sm.threads[parity], &count = sm.count[parity];
            if (mine >= bound) sm.who[atomicAdd(&threads, 1)] = static_cast<uint16_t>(tid);
            if (tid == 0) sm.threads[parity ^ 1] = sm.count[parity ^ 1] = 0;
            __syncthreads();
            // a thread's pieces to as many lanes, a warp's at most
            const int pieces = static_cast<int>(part.c1 - part.c0) * kPieces, all = threads;
            const int shift = pieces > 16 ? 5 : (pieces > 8 ? 4 : (pieces > 4 ? 3 : 2));
            for (int w = tid >> shift; w < all; w += kThreads >> shift) {
                const int i0 = part.first_of(part.c0) + (sm.who[w] - tid) * VEC;
#pragma unroll 4
                for (int j = tid & ((1 << shift) - 1); j < pieces; j += 1 << shift) {
                    const int i = i0 + j * (kThreads * VEC);
                    float v[VEC];
                    if (i >= 0 && i + VEC <= p.V) {
                        unpack(*reinterpret_cast<const uint4*>(part.x + i), v, T());
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            v[e] = i + e >= 0 && i + e < p.V ? as_float(part.x[i + e]) : -INFINITY;
                    }
                    float mx = v[0];
#pragma unroll
                    for (int e = 1; e < VEC; e += 2) mx = max3(mx, v[e], v[e + 1 < VEC ? e + 1 : e]);
                    if (mx < bound) continue;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        if (v[e] >= bound) {
                            const int at = atomicAdd(&count, 1);
                            if (at < kList) top.list[at] = key_of(v[e], static_cast<uint32_t>(i + e));
                        }
                    }
                }
            }
            __syncthreads();
            int n = count;
            if (n <= 2 * 32) {
                if (warp == 0) kept = first_of_few(top, n, p.k, lane);
            } else {
                if (n > kList)
                    n = careful(top, sm, count, part.x, max(part.first_of(part.c0) - tid * VEC, 0),
                                min(part.first_of(part.c1) - tid * VEC, p.V), p.k);
                kept = first_of_list(top, sm, n, p.k);
            }
        }
        if (ctas > 1) {
            // (the first has begun, and is done with the row before)
            cluster.barrier_wait();
            if (tid == 0) *cluster.map_shared_rank(&sm.all[rank], 0) = st;
            // (empty places: keys below all others, no two equal)
            if (TOP && tid < p.k) {
                const uint32_t i = rank * p.k + tid;
                cluster.map_shared_rank(&top, 0)->far[i] = tid < kept ? top.best[tid] : i;
            }
            cluster.barrier_arrive();
            if (rank == 0) {
                cluster.barrier_wait();
                if (warp == 0) {
                    st = {-INFINITY, 0.0f, 0.0f, 0};
                    if (lane < ctas) st = sm.all[lane];
                    st = warp_join(st);
                }
                if (TOP) {
                    put_in_order(top.best, top.far, static_cast<int>(ctas) * p.k, p.k);
                }
                cluster.barrier_arrive();
            } else {
                cluster.barrier_wait();
                cluster.barrier_arrive();
            }
        } else if (TOP) {
            if (tid >= kept && tid < p.k) top.best[tid] = 0;
        }
        if (rank == 0 && warp == 0) {
            // nothing but -inf: no distribution, the sum is 0. A NaN or +inf: the sum is NaN.
            __syncwarp();
            const bool given = tok >= 0 && tok < p.V;
            const float logl = logf(st.l);
            const bool bad = !(st.l >= 0.0f);
            auto logp = [&](float x) { return x == -INFINITY && !bad ? -INFINITY : x - st.m - logl; };
            if (lane == 0) {
                p.lp[row] = given ? logp(xt) : NAN;
                if (p.ranks) p.ranks[row] = given && !bad ? st.above : -1;
                if (p.entropy) p.entropy[row] = st.l == 0.0f ? 0.0f : logl - st.s / st.l;
            }
            if (TOP) {
                const uint64_t key = lane < p.k ? top.best[lane] : 0ull;
                const int found = __popc(__ballot_sync(0xffffffffu, (key >> 32) != 0));
                int id = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
                float value = unordered(static_cast<uint32_t>(key >> 32));
                if (found < p.k) {
                    // fewer finite values than alternatives: -inf ones follow, of which at
                    // least k - found lie among the first 64 values (or among all)
                    const bool a = lane < p.V && as_float(part.x[lane]) == -INFINITY;
                    const bool b = lane + 32 < p.V && as_float(part.x[lane + 32]) == -INFINITY;
                    const uint32_t lo = __ballot_sync(0xffffffffu, a), hi = __ballot_sync(0xffffffffu, b);
                    if (lane >= found) {
                        uint64_t left = static_cast<uint64_t>(hi) << 32 | lo;
                        for (int i = found; i < lane; ++i) left &= left - 1;
                        id = __ffsll(static_cast<long long>(left)) - 1;
                        value = -INFINITY;
                    }
                }
                if (lane < p.k) {
                    p.top_ids[row * p.k + lane] = bad ? -1 : id;
                    p.top_lp[row * p.k + lane] = bad ? NAN : logp(value);
                }
            }
        }
        tok = tok_next;
        xt = xt_next;
    }
    if (ctas > 1) cluster.barrier_wait();
}

template <typename T, bool TOP>
cudaError_t launch(const LogprobParams& p, int64_t clusters, int ctas, cudaStream_t st)
{
    const size_t smem = kStages * kSlot + (TOP ? sizeof(TopSmem) : 0);
    const cudaError_t e = cudaFuncSetAttribute(token_logprobs_kernel<T, TOP>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(clusters * ctas));
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
    PA_REQUIRE(V <= 0x7FFFFFFF - (1 << 16) && num_rows <= 0x7FFFFFFF, PA_ERR_UNSUPPORTED,
               "%s: too many rows or tokens", name);
    PA_REQUIRE(aligned(logits, dtype == PA_DTYPE_F32 ? 4 : 2) && aligned(tokens, token_type == PA_INDEX_I64 ? 8 : 4) &&
                   aligned(logprobs, 4) && aligned(ranks, 4) && aligned(entropy, 4) &&
                   (top == 0 || (aligned(top_ids, 4) && aligned(top_logprobs, 4))),
               PA_ERR_INVALID, "%s: misaligned pointer", name);
    if (num_rows == 0) return PA_OK;
    // (rows are read while others' results are already written, and read again)
    struct Range { const void* at; uint64_t bytes; };
    const uint64_t r4 = 4ull * num_rows;
    const Range in[] = {{logits, ((num_rows - 1) * static_cast<uint64_t>(row_stride) + V) * (dtype == PA_DTYPE_F32 ? 4 : 2)},
                        {tokens, r4 * (token_type == PA_INDEX_I64 ? 2 : 1)}};
    const Range out[] = {{logprobs, r4}, {ranks, ranks ? r4 : 0}, {entropy, entropy ? r4 : 0},
                         {top_ids, top ? r4 * top : 0}, {top_logprobs, top ? r4 * top : 0}};
    for (const Range& o : out) {
        for (const Range& i : in)
            PA_REQUIRE(!overlap(o.at, o.bytes, i.at, i.bytes), PA_ERR_INVALID, "%s: an output overlaps an input", name);
        for (const Range& i : out)
            PA_REQUIRE(&i == &o || !overlap(o.at, o.bytes, i.at, i.bytes), PA_ERR_INVALID, "%s: outputs overlap", name);
    }
    const int sms = device_sm_count();
    PA_REQUIRE(sms > 0, PA_ERR_CUDA, "%s: cannot query the device", name);
    LogprobParams p;
    p.x = logits;
    p.stride = num_rows > 1 ? row_stride : 0;
    p.tok = tokens;
    p.tok_type = token_type;
    p.R = num_rows;
    p.V = V;
    p.k = top;
    p.lp = logprobs;
    p.ranks = ranks;
    p.entropy = entropy;
    p.top_ids = top_ids;
    p.top_lp = top_logprobs;
    // As many CTAs a row as there is room for, two an SM, and as have a chunk each. (Clusters
    // do not fill every group of SMs: 36 of 8 CTAs run at once on 152 SMs, 74 of 4, all 152
    // of 2. 38 rows x 131072 took 22.7 us on clusters of 8, 14.4 on those of 4.)
    const int chunk = kThreads * kPieces * 16 / (dtype == PA_DTYPE_F32 ? 4 : 2);
    int ctas = kMaxCluster;
    while (ctas > 1 && (num_rows * ctas > 2 * sms - (ctas > 2 ? 2 * ctas : 0) || V <= chunk * (ctas / 2))) ctas /= 2;
    const int64_t clusters = std::min<int64_t>(num_rows, 2 * sms / ctas);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == PA_DTYPE_F32) e = top ? launch<float, true>(p, clusters, ctas, st) : launch<float, false>(p, clusters, ctas, st);
    else e = top ? launch<__nv_bfloat16, true>(p, clusters, ctas, st) : launch<__nv_bfloat16, false>(p, clusters, ctas, st);
    PA_REQUIRE(e == cudaSuccess, PA_ERR_CUDA, "%s: launch: %s", name, cudaGetErrorString(e));
    return check_launch(name);
}

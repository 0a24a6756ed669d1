// plan.cu -- block tables, slots and positions of a step's tokens from the
// requests' lengths, on the GPU.
//
// With a = kv_act_seqs[b] and n = new_lens[b]: cu is the running sum of n, a
// request needs ceil((a + n) / BS) - ceil(a / BS) new blocks, which it takes from
// the pool behind those of the requests before it, so the running sum of the needs
// says which. Token i's slot then is its position's block, an old or a new one, and
// the place in it.
//
// A few kilobytes: bound by the launch and a chain of four dependent steps (lengths,
// the two sums, block ids, slots). Every CTA takes the sums of all requests anew, two
// requests a thread, rather than wait for another's or for another launch; the
// tokens and the new blocks are dealt to the CTAs' threads, each of which finds its
// request by bisection in shared memory. 64 requests of a token each take 6.2 us launched
// by the host and 3.8 one after another in a graph, 1000 requests, 250 of them with a
// prompt's chunk, in 65536 rows 6.3 and 5.1.
#include "common.cuh"

#include <algorithm>

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxB = 1024;
constexpr int kPer = kMaxB / kThreads;       // requests a thread
constexpr int kTokens = 1024;                // tokens a CTA

struct PlanParams {
    const int *act, *lens, *pool, *head;
    int* bt;
    void* slots;
    int slot_type;
    int *pos, *batch, *cu, *new_act, *new_head;
    int64_t num_blocks;
    int B, T, P, width, BS;
};

// The first index in [0, n) whose value is above x, n if there is none (v ascending).
__device__ __forceinline__ int first_above(const int* v, int n, int x)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ int blocks_of(int positions, int BS) { return positions / BS + (positions % BS != 0); }

__global__ void __launch_bounds__(kThreads) plan_batch_kernel(const PlanParams p)
{
    // cu: rows up to and with each request's; ends: new blocks up to and with its own
    // (both cut to 31 bits); held: positions before the step, ~ of them if refused
    __shared__ int cu[kMaxB], ends[kMaxB], held[kMaxB];
    __shared__ int64_t sums[2][kThreads / 32];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = min(max(__ldg(p.head), 0), p.P);
    int64_t a[kPer], n[kPer], rows = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * kPer + i;
        a[i] = b < p.B ? max(__ldg(p.act + b), 0) : 0;
        n[i] = b < p.B ? max(__ldg(p.lens + b), 0) : 0;
        rows += n[i];
    }
    if (tid == 0) last = 0;
    // a sum over all threads before this one, 64 bits: lengths are not bounded
    auto before = [&](int64_t mine, int which) {
        int64_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sums[which][warp] = x;
        __syncthreads();
        x -= mine;
        for (int w = 0; w < warp; ++w) x += sums[which][w];
        return x;
    };
    int64_t row = before(rows, 0), need[kPer], needs = 0;
    bool fits[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        row += n[i];
        fits[i] = a[i] + n[i] <= static_cast<int64_t>(p.width) * p.BS && row <= p.T;
        need[i] = fits[i] ? (a[i] + n[i] + p.BS - 1) / p.BS - (a[i] + p.BS - 1) / p.BS : 0;
        needs += need[i];
        if (tid * kPer + i < p.B) cu[tid * kPer + i] = static_cast<int>(min(row, static_cast<int64_t>(p.T)));
    }
    int64_t end = before(needs, 1);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * kPer + i;
        end += need[i];
        fits[i] = fits[i] && (need[i] == 0 || head + end <= p.P);
        if (b >= p.B) continue;
        ends[b] = static_cast<int>(min(end, static_cast<int64_t>(0x7FFFFFFF)));
        held[b] = fits[i] ? static_cast<int>(a[i]) : ~static_cast<int>(a[i]);
        // (those that fit and need blocks are the first of those that need blocks)
        if (fits[i] && need[i] > 0) atomicMax(&last, static_cast<int>(end));
        if (blockIdx.x == 0) {
            p.cu[b + 1] = cu[b];
            p.new_act[b] = static_cast<int>(fits[i] ? a[i] + n[i] : a[i]);
        }
    }
    __syncthreads();
    const int blocks = last, real = p.B > 0 ? cu[p.B - 1] : 0;
    if (blockIdx.x == 0 && tid == 0) {
        p.cu[0] = 0;
        *p.new_head = head + blocks;
    }
    const int64_t step = gridDim.x * kThreads, first = blockIdx.x * kThreads + tid;
    // ---- the new blocks' entries ----
    for (int64_t i = first; i < blocks; i += step) {
        const int e = static_cast<int>(i), b = first_above(ends, p.B, e);
        const int at = blocks_of(held[b], p.BS) + (e - (b > 0 ? ends[b - 1] : 0));
        p.bt[static_cast<int64_t>(b) * p.width + at] = __ldg(p.pool + head + e);
    }
    // ---- the tokens ----
    for (int64_t i = first; i < p.T; i += step) {
        const int t = static_cast<int>(i);
        int b = 0, pos = 0;
        int64_t slot = -1;
        if (t < real) {
            b = first_above(cu, p.B, t);
            const bool ok = held[b] >= 0;
            const int at = ok ? held[b] : ~held[b];
            // (a refused request's may pass 31 bits: cut)
            pos = static_cast<int>(min(static_cast<int64_t>(at) + t - (b > 0 ? cu[b - 1] : 0),
                                       static_cast<int64_t>(0x7FFFFFFF)));
            if (ok) {
                const int have = blocks_of(at, p.BS), j = pos / p.BS;
                const int block = j < have ? __ldg(p.bt + static_cast<int64_t>(b) * p.width + j)
                                           : __ldg(p.pool + head + (b > 0 ? ends[b - 1] : 0) + (j - have));
                if (block >= 0 && block < p.num_blocks) slot = static_cast<int64_t>(block) * p.BS + (pos - j * p.BS);
            }
        }
        p.pos[t] = pos;
        p.batch[t] = b;
        if (p.slot_type == PA_INDEX_I64) static_cast<int64_t*>(p.slots)[t] = slot;
        else static_cast<int*>(p.slots)[t] = static_cast<int>(slot);
    }
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_plan_batch(const int32_t* kv_act_seqs, const int32_t* new_lens, const int32_t* pool,
                                   const int32_t* pool_head, int32_t* block_table, void* slot_mapping, int slot_type,
                                   int32_t* positions, int32_t* token_batch, int32_t* cu_tokens,
                                   int32_t* new_act_seqs, int32_t* new_pool_head, int B, int64_t num_tokens,
                                   int64_t pool_size, int64_t num_blocks, int block_size, int max_blocks_per_seq,
                                   void* stream)
{
    const char* name = "pa_plan_batch";
    PA_REQUIRE(B >= 0 && num_tokens >= 0 && pool_size >= 0 && num_blocks > 0 && block_size > 0 &&
                   max_blocks_per_seq > 0,
               PA_ERR_INVALID, "%s: empty or negative size", name);
    PA_REQUIRE(cu_tokens && pool_head && new_pool_head &&
                   (B == 0 || (kv_act_seqs && new_lens && block_table && new_act_seqs)) && (pool_size == 0 || pool) &&
                   (num_tokens == 0 || (slot_mapping && positions && token_batch)),
               PA_ERR_NULLPTR, "%s: NULL tensor pointer", name);
    PA_REQUIRE(slot_type == PA_INDEX_I32 || slot_type == PA_INDEX_I64, PA_ERR_INVALID, "%s: unknown slot type %d", name,
               slot_type);
    PA_REQUIRE(B <= kMaxB, PA_ERR_UNSUPPORTED, "%s: batch %d > %d", name, B, kMaxB);
    PA_REQUIRE(num_tokens <= 0x7FFFFFFF && pool_size <= 0x7FFFFFFF &&
                   static_cast<int64_t>(max_blocks_per_seq) * block_size <= 0x7FFFFFFF && block_size <= (1 << 30),
               PA_ERR_UNSUPPORTED, "%s: tokens, pool or positions of 2^31 or more", name);
    PA_REQUIRE(slot_type == PA_INDEX_I64 || num_blocks <= 0x7FFFFFFF / block_size, PA_ERR_UNSUPPORTED,
               "%s: slots of 2^31 or more (use int64)", name);
    for (const void* x : {static_cast<const void*>(kv_act_seqs), static_cast<const void*>(new_lens),
                          static_cast<const void*>(pool), static_cast<const void*>(pool_head),
                          static_cast<const void*>(block_table), static_cast<const void*>(positions),
                          static_cast<const void*>(token_batch), static_cast<const void*>(cu_tokens),
                          static_cast<const void*>(new_act_seqs), static_cast<const void*>(new_pool_head)})
        PA_REQUIRE(aligned(x, 4), PA_ERR_INVALID, "%s: misaligned pointer", name);
    PA_REQUIRE(aligned(slot_mapping, slot_type == PA_INDEX_I64 ? 8 : 4), PA_ERR_INVALID, "%s: misaligned slot_mapping",
               name);
    // every CTA reads all inputs while others already write
    struct Range { const void* at; uint64_t bytes; };
    const uint64_t b4 = 4ull * B, t4 = 4ull * num_tokens;
    const Range in[] = {{kv_act_seqs, b4}, {new_lens, b4}, {pool, 4ull * pool_size}, {pool_head, 4}};
    const Range out[] = {{block_table, b4 * max_blocks_per_seq},
                         {slot_mapping, t4 * (slot_type == PA_INDEX_I64 ? 2 : 1)},
                         {positions, t4}, {token_batch, t4}, {cu_tokens, b4 + 4}, {new_act_seqs, b4},
                         {new_pool_head, 4}};
    for (const Range& o : out) {
        for (const Range& i : in)
            PA_REQUIRE(!overlap(o.at, o.bytes, i.at, i.bytes), PA_ERR_INVALID, "%s: an output overlaps an input", name);
        for (const Range& i : out)
            PA_REQUIRE(&i == &o || !overlap(o.at, o.bytes, i.at, i.bytes), PA_ERR_INVALID,
                       "%s: outputs overlap", name);
    }
    const int sms = device_sm_count();
    PA_REQUIRE(sms > 0, PA_ERR_CUDA, "%s: cannot query the device", name);
    PlanParams p;
    p.act = kv_act_seqs;
    p.lens = new_lens;
    p.pool = pool;
    p.head = pool_head;
    p.bt = block_table;
    p.slots = slot_mapping;
    p.slot_type = slot_type;
    p.pos = positions;
    p.batch = token_batch;
    p.cu = cu_tokens;
    p.new_act = new_act_seqs;
    p.new_head = new_pool_head;
    p.num_blocks = num_blocks;
    p.B = B;
    p.T = static_cast<int>(num_tokens);
    p.P = static_cast<int>(pool_size);
    p.width = max_blocks_per_seq;
    p.BS = block_size;
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>((num_tokens + kTokens - 1) / kTokens, sms));
    plan_batch_kernel<<<static_cast<unsigned>(ctas), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return check_launch(name);
}

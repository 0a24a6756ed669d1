// draft.cu -- verification of drafted tokens against the target's
// probabilities, and the accepted branch kept in the paged cache.
#include "common.cuh"

#include <cooperative_groups.h>

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxNodes = 1024;

// ---- verification ------------------------------------------------------------------
// One cluster of kVC CTAs per sequence; every thread follows the same walk
// over the nodes. A node's first test needs three values (p, q and u at its
// token), gathered for all nodes at once ahead of the walk. A rejection of a
// drawn draft needs all of R = max(R - z Q, 0) and its sum, and the draw at
// the end needs R: CTA r keeps channels [r, r + 1) * slice of R in shared
// memory, warp w of it the w-th segment of the slice, in index order, so that
// the draw needs the 128 segments' sums and then one segment's 32-wide steps.
// The weights are 2^-45 integers: their sums are exact, so the drawn index
// depends neither on the number of CTAs nor on the order of summation.
// Bound by the rows of p and q read (one or two of V floats per sequence) on
// large batches, by the chain launch, gather, row, two cluster barriers on
// small ones.
constexpr int kVC = 8;
constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kSegs = kVC * kVWarps;
constexpr int kMaxV = 1 << 18;

struct VerifyParams {
    const float *p, *q;
    const int *tok, *par;
    const float* u;
    const int* len;
    int S1, V, slice, seg;
    int *accepted, *path, *tokens;
};

// floor(min(r, 1) * 2^45) for r > 0, 0 for the rest and for NaN.
__device__ __forceinline__ unsigned long long weight(float r)
{
    if (!(r > 0.0f)) return 0;
    const uint32_t u = __float_as_uint(fminf(r, 1.0f));
    const int sh = static_cast<int>(u >> 23) - 105;      // exponent - 127 - 23 + 45
    const unsigned long long m = (u & 0x7FFFFFu) | 0x800000u;
    return sh >= 0 ? m << sh : (sh > -24 ? m >> -sh : 0ull);
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct VerifySmem {
    double p0[kMaxNodes], q0[kMaxNodes];
    float u[kMaxNodes];
    int par[kMaxNodes], tok[kMaxNodes];
    unsigned long long wsum[kVWarps];
    unsigned long long all[kSegs];
};

__global__ void __cluster_dims__(kVC, 1, 1) __launch_bounds__(kVThreads) tree_verify_kernel(const VerifyParams a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    VerifySmem& sm = *reinterpret_cast<VerifySmem*>(raw);
    float* R = reinterpret_cast<float*>(raw + sizeof(VerifySmem));
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cl.block_rank());
    const int64_t b = blockIdx.x / kVC;
    int* path = a.path + b * a.S1;
    int* tokens = a.tokens + b * a.S1;
    int n = a.len ? __ldg(a.len + b) : a.S1;
    n = n < 0 ? 0 : (n > a.S1 ? a.S1 : n);
    if (n == 0) {                                         // the whole cluster
        if (rank == 0) {
            for (int i = tid; i < a.S1; i += kVThreads) path[i] = tokens[i] = -1;
            if (tid == 0) a.accepted[b] = 0;
        }
        return;
    }
    const float* pb = a.p + b * a.S1 * a.V;
    const float* qb = a.q ? a.q + b * a.S1 * a.V : nullptr;
    for (int s = tid; s < n; s += kVThreads) {
        const int par = __ldg(a.par + b * a.S1 + s), x = __ldg(a.tok + b * a.S1 + s);
        const bool ok = s > 0 && par >= 0 && par < s && x >= 0 && x < a.V;
        sm.par[s] = ok ? par : -1;
        sm.tok[s] = x;
        sm.u[s] = __ldg(a.u + b * a.S1 + s);
        const int64_t at = static_cast<int64_t>(ok ? par : 0) * a.V + (ok ? x : 0);
        sm.p0[s] = ok ? static_cast<double>(__ldg(pb + at)) : 0.0;
        sm.q0[s] = ok ? (qb ? static_cast<double>(__ldg(qb + at)) : 1.0) : 0.0;
    }
    __syncthreads();

    // this warp's channels of R: [lo, hi) of the vocabulary, R[lo - base ..]
    const int base = rank * a.slice;
    const int lo = min(base + warp * a.seg, min(base + a.slice, a.V));
    const int hi = min(lo + a.seg, min(base + a.slice, a.V));
    // R of node `cur` from p, or one rejection further, and the segments' sums
    auto sums = [&](unsigned long long mine) {
        mine = warp_sum(mine);
        if (lane == 0) sm.wsum[warp] = mine;
        cl.sync();
        if (tid < kSegs) sm.all[tid] = cl.map_shared_rank(sm.wsum, tid / kVWarps)[tid % kVWarps];
        __syncthreads();
        unsigned long long z = 0;
        for (int i = lane; i < kSegs; i += 32) z += sm.all[i];
        return warp_sum(z);
    };
    auto load = [&](int cur) {
        unsigned long long w = 0;
        const float* src = pb + static_cast<int64_t>(cur) * a.V;
#pragma unroll 8
        for (int i = lo + lane; i < hi; i += 32) {
            const float r = __ldg(src + i);
            R[i - base] = r;
            w += weight(r);
        }
        return w;
    };

    int cur = 0, acc = 1;
    bool held = false, summed = false;   // R holds cur's rest; sm.all its sums
    double z = 1.0;
    unsigned long long Z = 0;
    for (int s = 1; s < n; ++s) {
        if (sm.par[s] != cur) continue;
        const int x = sm.tok[s];
        double rx = sm.p0[s];
        if (qb) {
            if (held) rx = static_cast<double>(*cl.map_shared_rank(R + x % a.slice, x / a.slice));
        } else {
            for (int t = cur + 1; t < s; ++t)
                if (sm.par[t] == cur && sm.tok[t] == x) rx = 0.0;   // rejected before: R(x) is 0
        }
        if (static_cast<double>(sm.u[s]) * z * sm.q0[s] < rx) {
            if (rank == 0 && tid == 0) {
                path[acc] = s;
                tokens[acc - 1] = x;
            }
            ++acc;
            cur = s;
            held = summed = false;
            z = 1.0;
        } else if (qb) {
            const float zf = static_cast<float>(z);
            const float* src = pb + static_cast<int64_t>(cur) * a.V;
            const float* qr = qb + static_cast<int64_t>(cur) * a.V;
            cl.sync();                    // every thread has read R(x)
            unsigned long long w = 0;
#pragma unroll 8
            for (int i = lo + lane; i < hi; i += 32) {
                const float r0 = held ? R[i - base] : __ldg(src + i);
                const float r = fmaxf(__fsub_rn(r0, __fmul_rn(zf, __ldg(qr + i))), 0.0f);
                R[i - base] = r;
                w += weight(r);
            }
            Z = sums(w);
            held = summed = true;
            z = static_cast<double>(static_cast<float>(static_cast<double>(Z) * 0x1p-45));
        } else {
            z -= rx;
        }
    }
    // ---- the draw ----
    if (!summed) {
        cl.sync();                        // sm.wsum and R of an earlier node are not read any more
        unsigned long long w = load(cur);
        if (!qb) {
            // tokens of cur's children, all of them rejected, are out
            __syncwarp();
            for (int t = cur + 1; t < n; ++t)
                if (sm.par[t] == cur && sm.tok[t] >= lo && sm.tok[t] < hi) {
                    if (lane == (sm.tok[t] - lo) % 32) {
                        w -= weight(R[sm.tok[t] - base]);
                        R[sm.tok[t] - base] = 0.0f;
                    }
                    __syncwarp();
                }
        }
        Z = sums(w);
    }
    if (Z == 0) {
        cl.sync();
        Z = sums(load(cur));
    }
    if (rank == 0) {
        if (tid == 0) {
            a.accepted[b] = acc;
            path[0] = 0;
            if (Z == 0) tokens[acc - 1] = -1;
        }
        for (int i = acc + tid; i < a.S1; i += kVThreads) path[i] = tokens[i] = -1;
    }
    if (Z != 0) {
        const float u0 = sm.u[0];
        unsigned long long t = u0 > 0.0f ? static_cast<unsigned long long>(static_cast<double>(u0) * static_cast<double>(Z)) : 0ull;
        if (t >= Z) t = Z - 1;
        unsigned long long before = 0;
        const int mine = rank * kVWarps + warp;
        for (int i = lane; i < mine; i += 32) before += sm.all[i];
        before = warp_sum(before);
        if (t >= before && t - before < sm.all[mine]) {
            for (int i0 = lo; i0 < hi; i0 += 32) {
                const int i = i0 + lane;
                unsigned long long c = i < hi ? weight(R[i - base]) : 0ull;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned long long up = __shfl_up_sync(0xffffffffu, c, o);
                    if (lane >= o) c += up;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, before + c > t);
                if (hit) {
                    if (lane == 0) tokens[acc - 1] = i0 + __ffs(static_cast<int>(hit)) - 1;
                    break;
                }
                before += __shfl_sync(0xffffffffu, c, 31);
            }
        }
    }
    cl.sync();                            // no CTA leaves while another reads its shared memory
}

// ---- the accepted branch in the cache ------------------------------------------------
// One CTA per (sequence, group of heads); a thread owns one 16-byte chunk of
// one head's K or V (or one key scale) and moves it for the branch's nodes in
// order. path[i] >= i, so a node's chunk is read before the move that
// overwrites it comes, and only this thread touches it: no barrier between
// loads and stores. Latency-bound: a chain of four dependent loads.
constexpr int kKThreads = 256;
constexpr int kKBatch = 8;

struct KeepParams {
    uint8_t *kc, *vc;
    float* ks;
    const int *bt, *act, *len, *path, *accepted;
    int* new_act;
    int S1, H, chunks, BS;
    int64_t num_blocks;
    int max_blocks, layout, heads_per_cta;
};

__global__ void __launch_bounds__(kKThreads) cache_keep_path_kernel(const KeepParams p)
{
    __shared__ int64_t src[kMaxNodes], dst[kMaxNodes];   // token slots, src -1: no move
    const int b = blockIdx.x, tid = threadIdx.x;
    const int act = max(__ldg(p.act + b), 0);
    int n = p.len ? __ldg(p.len + b) : p.S1;
    n = n < 0 ? 0 : (n > p.S1 ? p.S1 : n);
    n = min(n, act);
    int m = __ldg(p.accepted + b);
    m = m < 0 ? 0 : (m > n ? n : m);
    const int ctx = act - n;
    if (blockIdx.y == 0 && tid == 0) p.new_act[b] = ctx + m;
    auto slot = [&](int pos) -> int64_t {
        const int bi = pos / p.BS;
        if (pos < 0 || bi >= p.max_blocks) return -1;
        const int id = __ldg(p.bt + static_cast<int64_t>(b) * p.max_blocks + bi);
        return id >= 0 && id < p.num_blocks ? static_cast<int64_t>(id) * p.BS + pos % p.BS : -1;
    };
    for (int i = tid; i < m; i += kKThreads) {
        const int s = __ldg(p.path + static_cast<int64_t>(b) * p.S1 + i);
        int64_t from = -1, to = -1;
        if (s != i && s >= 0 && s < n) {
            from = slot(ctx + s);
            to = slot(ctx + i);
        }
        src[i] = to >= 0 ? from : -1;
        dst[i] = to;
    }
    __syncthreads();
    const int h0 = blockIdx.y * p.heads_per_cta;
    const int heads = min(p.heads_per_cta, p.H - h0);
    const int per = 2 * p.chunks;
    for (int c = tid; c < heads * (per + 1); c += kKThreads) {
        const int h = h0 + c / (per + 1), k = c % (per + 1);
        auto row = [&](int64_t slot_) { return cache_row(p.layout, slot_ / p.BS, slot_ % p.BS, h, p.BS, p.H); };
        if (k == per) {
            for (int i = 0; i < m; ++i)
                if (src[i] >= 0) p.ks[row(dst[i])] = p.ks[row(src[i])];
            continue;
        }
        uint4* base = reinterpret_cast<uint4*>(k < p.chunks ? p.kc : p.vc) + (k < p.chunks ? k : k - p.chunks);
        for (int i0 = 0; i0 < m; i0 += kKBatch) {
            uint4 v[kKBatch];
#pragma unroll
            for (int j = 0; j < kKBatch; ++j)
                if (i0 + j < m && src[i0 + j] >= 0) v[j] = base[row(src[i0 + j]) * p.chunks];
#pragma unroll
            for (int j = 0; j < kKBatch; ++j)
                if (i0 + j < m && src[i0 + j] >= 0) base[row(dst[i0 + j]) * p.chunks] = v[j];
        }
    }
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_tree_verify(const float* target_probs, const float* draft_probs,
                                    const int32_t* draft_tokens, const int32_t* parents,
                                    const float* uniforms, const int32_t* tree_len, int B, int S1, int V,
                                    int32_t* accepted, int32_t* path, int32_t* tokens, void* stream)
{
    PA_REQUIRE(target_probs && draft_tokens && parents && uniforms && accepted && path && tokens,
               PA_ERR_NULLPTR, "pa_tree_verify: NULL tensor pointer");
    PA_REQUIRE(B >= 0 && S1 > 0 && V > 0, PA_ERR_INVALID, "pa_tree_verify: empty or negative size");
    PA_REQUIRE(S1 <= kMaxNodes, PA_ERR_UNSUPPORTED, "pa_tree_verify: S1 %d > %d", S1, kMaxNodes);
    PA_REQUIRE(V <= kMaxV, PA_ERR_UNSUPPORTED, "pa_tree_verify: V %d > %d", V, kMaxV);
    PA_REQUIRE(B <= (1 << 24), PA_ERR_UNSUPPORTED, "pa_tree_verify: batch %d > %d", B, 1 << 24);
    const void* ptrs[] = {target_probs, draft_probs, draft_tokens, parents, uniforms, tree_len, accepted, path, tokens};
    for (const void* q : ptrs)
        PA_REQUIRE(aligned(q, 4), PA_ERR_INVALID, "pa_tree_verify: misaligned pointer");
    if (B == 0) return PA_OK;
    VerifyParams a;
    a.p = target_probs;
    a.q = draft_probs;
    a.tok = draft_tokens;
    a.par = parents;
    a.u = uniforms;
    a.len = tree_len;
    a.S1 = S1;
    a.V = V;
    a.seg = (V + kSegs * 32 - 1) / (kSegs * 32) * 32;
    a.slice = a.seg * kVWarps;
    a.accepted = accepted;
    a.path = path;
    a.tokens = tokens;
    const size_t smem = sizeof(VerifySmem) + static_cast<size_t>(a.slice) * sizeof(float);
    // (per device: set on every call, a host-side table write)
    cudaError_t e = cudaFuncSetAttribute(tree_verify_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    PA_REQUIRE(e == cudaSuccess, PA_ERR_CUDA, "pa_tree_verify: smem attribute: %s", cudaGetErrorString(e));
    tree_verify_kernel<<<static_cast<unsigned>(B) * kVC, kVThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
    return check_launch("pa_tree_verify");
}

extern "C" pa_status pa_fp8_cache_keep_path(void* key_cache, void* value_cache, float* key_scale_cache,
                                            const int32_t* block_table, const int32_t* kv_act_seqs,
                                            const int32_t* tree_len, const int32_t* path,
                                            const int32_t* accepted, int32_t* new_act_seqs, int B, int S1,
                                            int NKV, int head_size, int block_size, int64_t num_blocks,
                                            int max_blocks_per_seq, int layout, void* stream)
{
    const char* name = "pa_fp8_cache_keep_path";
    PA_REQUIRE(key_cache && value_cache && key_scale_cache && block_table && kv_act_seqs && path &&
                   accepted && new_act_seqs,
               PA_ERR_NULLPTR, "%s: NULL tensor pointer", name);
    PA_REQUIRE(B >= 0 && S1 > 0 && NKV > 0 && head_size > 0 && block_size > 0 && num_blocks > 0 &&
                   max_blocks_per_seq > 0,
               PA_ERR_INVALID, "%s: empty or negative size", name);
    PA_REQUIRE(layout == PA_LAYOUT_BSND || layout == PA_LAYOUT_BNBD, PA_ERR_INVALID,
               "%s: unknown layout %d", name, layout);
    PA_REQUIRE(S1 <= kMaxNodes, PA_ERR_UNSUPPORTED, "%s: S1 %d > %d", name, S1, kMaxNodes);
    PA_REQUIRE(head_size % 16 == 0, PA_ERR_UNSUPPORTED, "%s: head_size %d is not a multiple of 16", name,
               head_size);
    PA_REQUIRE(new_act_seqs != kv_act_seqs, PA_ERR_INVALID,
               "%s: new_act_seqs must be another buffer than kv_act_seqs", name);
    PA_REQUIRE(aligned(key_cache, 16) && aligned(value_cache, 16) && aligned(key_scale_cache, 4), PA_ERR_INVALID,
               "%s: misaligned pointer", name);
    if (B == 0) return PA_OK;
    KeepParams p;
    p.kc = static_cast<uint8_t*>(key_cache);
    p.vc = static_cast<uint8_t*>(value_cache);
    p.ks = key_scale_cache;
    p.bt = block_table;
    p.act = kv_act_seqs;
    p.len = tree_len;
    p.path = path;
    p.accepted = accepted;
    p.new_act = new_act_seqs;
    p.S1 = S1;
    p.H = NKV;
    p.chunks = head_size / 16;
    p.BS = block_size;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.layout = layout;
    const int per = 2 * p.chunks + 1;
    p.heads_per_cta = kKThreads / per > 0 ? kKThreads / per : 1;
    const int64_t gy = (NKV + p.heads_per_cta - 1) / p.heads_per_cta;
    PA_REQUIRE(gy <= 65535, PA_ERR_UNSUPPORTED, "%s: too many heads (%d)", name, NKV);
    cache_keep_path_kernel<<<dim3(static_cast<unsigned>(B), static_cast<unsigned>(gy)), kKThreads, 0,
                             static_cast<cudaStream_t>(stream)>>>(p);
    return check_launch(name);
}

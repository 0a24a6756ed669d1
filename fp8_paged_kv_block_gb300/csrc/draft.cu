// draft.cu -- verification of drafted tokens against the target's
// probabilities, and the accepted branch kept in the paged cache.
#include "common.cuh"

#include <cooperative_groups.h>

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxNodes = 1024;

// ---- verification ------------------------------------------------------------------
// One cluster of CTAs per sequence; every thread follows the same walk over the
// nodes. A node's tests need p, q and u at its token alone (R after k rejections
// is replayed from p, q and the z of each), gathered for all nodes at once ahead
// of the walk. A rejection of a drawn draft needs the sum of R over the
// vocabulary, and the draw at the end R's prefix sums: warp w of the cluster takes
// the w-th segment of the vocabulary, replays R there and sums it; the draw then
// needs the segments' sums and one segment's 128-wide steps.
// The weights are 2^-45 integers: their sums are exact, so the drawn index
// depends neither on the number of CTAs nor on the order of summation.
// Bound by the rows of p and q read (one or two of V floats per sequence, again
// from L2 for each further rejection) on large batches, by the chain launch,
// gather, row, cluster barrier on small ones.
// A sequence gets 8 CTAs while the batch's CTAs number at most kResident, half as
// many for twice the batch: more CTAs shorten the pass over a row, and cost
// launches and cluster barriers once they no longer all run at once. kResident
// 304, 608, 1216: 53, 44, 44 us on 64 sequences of 16 nodes x 131072, 97, 65, 68
// on 128 of them; 61, 46, 49 us on 256 of 5 x 50000, 44, 36, 42 on 128.
constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSegs = kMaxCluster * kVWarps;
constexpr int kMaxV = 1 << 18;
constexpr int kResident = 608;               // 4 CTAs on each of 152 SMs

struct VerifyParams {
    const float *p, *q;
    const int *tok, *par;
    const float* u;
    const int* len;
    int S1, V, seg;
    int *accepted, *path, *tokens;
};

// floor(min(r, 1) * 2^45), 0 for NaN and below 0, as its top 23 and low 23 bits:
// r 2^22 and the rest of it 2^23 are exact, and adding 2^23 toward zero leaves
// their integer parts in the mantissa. hi and lo collect the floats' bits; kBias
// taken off once for each (modulo 2^32, where the sums of 2^9 terms lie) leaves
// the sums.
constexpr uint32_t kBias = 0x4B000000u;      // the bits of 2^23

__device__ __forceinline__ void add_weight(float r, uint32_t& hi, uint32_t& lo)
{
    const float x = fminf(fmaxf(r, 0.0f), 1.0f) * 0x1p22f;
    const float t = __fadd_rz(x, 0x1p23f);
    const float rest = x - (t - 0x1p23f);
    hi += __float_as_uint(t);
    lo += __float_as_uint(__fmaf_rz(rest, 0x1p23f, 0x1p23f));
}

__device__ __forceinline__ unsigned long long weight(float r)
{
    uint32_t hi = 0, lo = 0;
    add_weight(r, hi, lo);
    return (static_cast<unsigned long long>(hi - kBias) << 23) + (lo - kBias);
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct VerifySmem {
    unsigned long long all[2][kMaxSegs];     // the cluster's segments' sums, by pass parity
    // then, S1 long each: p and q at a node's token, u, the z's (two sets), parent, token
};

template <bool VEC>
__global__ void __launch_bounds__(kVThreads, 3) tree_verify_kernel(const VerifyParams a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    VerifySmem& sm = *reinterpret_cast<VerifySmem*>(raw);
    float* const p0 = reinterpret_cast<float*>(raw + sizeof(VerifySmem));
    float* const q0 = p0 + a.S1;
    float* const un = q0 + a.S1;
    float* const zs = un + a.S1;
    int* const par = reinterpret_cast<int*>(zs + 2 * a.S1);
    int* const tok = par + a.S1;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cl.block_rank()), ctas = static_cast<int>(cl.num_blocks());
    const int64_t b = blockIdx.x / ctas;
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
    // (no CTA writes into another's shared memory before that one has started)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const float* pb = a.p + b * a.S1 * a.V;
    const float* qb = a.q ? a.q + b * a.S1 * a.V : nullptr;
    for (int s = tid; s < n; s += kVThreads) {
        const int pr = __ldg(a.par + b * a.S1 + s), x = __ldg(a.tok + b * a.S1 + s);
        const bool ok = s > 0 && pr >= 0 && pr < s && x >= 0 && x < a.V;
        par[s] = ok ? pr : -1;
        tok[s] = x;
        un[s] = __ldg(a.u + b * a.S1 + s);
        const int64_t at = static_cast<int64_t>(ok ? pr : 0) * a.V + (ok ? x : 0);
        p0[s] = ok ? __ldg(pb + at) : 0.0f;
        q0[s] = ok ? (qb ? __ldg(qb + at) : 1.0f) : 0.0f;
    }
    __syncthreads();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");

    // this warp's segment [lo, hi) of the vocabulary
    const int segs = ctas * kVWarps, mine = rank * kVWarps + warp;
    const int lo = min(mine * a.seg, a.V), hi = min(lo + a.seg, a.V);
    const float* prow = pb;
    const float* qrow = qb;
    int cur = 0, acc = 1, rej = 0;           // current node, nodes accepted, drafts of cur rejected so far
    // The z's of cur's rejections. Every thread writes them, all the same, so that no
    // barrier is needed before they are read; a node's first takes the set that the
    // last node with rejections did not, as a slower warp may still be there (it has
    // passed that node's own cluster barrier, so no more than one set behind).
    float* zc = zs + a.S1;
    // R after `rej` rejections of drawn drafts, from p and q
    auto rest = [&](float r, float q) {
        for (int k = 0; k < rej; ++k) r = fmaxf(__fsub_rn(r, __fmul_rn(zc[k], q)), 0.0f);
        return r;
    };
    // R's weights summed over all of the vocabulary, and each segment's into sm.all
    int pass = 0;
    auto sums = [&](bool replay) {
        unsigned long long w = 0;
        if (VEC) {
#pragma unroll 2
            for (int i = lo + 4 * lane; i < hi; i += 128) {
                float4 r = __ldg(reinterpret_cast<const float4*>(prow + i));
                if (replay) {
                    const float4 q = __ldg(reinterpret_cast<const float4*>(qrow + i));
                    for (int k = 0; k < rej; ++k) {
                        const float z = zc[k];
                        r.x = fmaxf(__fsub_rn(r.x, __fmul_rn(z, q.x)), 0.0f);
                        r.y = fmaxf(__fsub_rn(r.y, __fmul_rn(z, q.y)), 0.0f);
                        r.z = fmaxf(__fsub_rn(r.z, __fmul_rn(z, q.z)), 0.0f);
                        r.w = fmaxf(__fsub_rn(r.w, __fmul_rn(z, q.w)), 0.0f);
                    }
                }
                uint32_t h = 0, l = 0;
                add_weight(r.x, h, l);
                add_weight(r.y, h, l);
                add_weight(r.z, h, l);
                add_weight(r.w, h, l);
                w += (static_cast<unsigned long long>(h - 4 * kBias) << 23) + (l - 4 * kBias);
            }
        } else {
#pragma unroll 4
            for (int i = lo + lane; i < hi; i += 32) {
                float r = __ldg(prow + i);
                if (replay) r = rest(r, __ldg(qrow + i));
                w += weight(r);
            }
        }
        if (!replay && !qb && rej > 0) {
            // tokens of cur's children, all of them rejected, are out (a repeated one
            // has p0 0)
            for (int t = cur + 1; t < n; ++t)
                if (lane == 0 && par[t] == cur && tok[t] >= lo && tok[t] < hi) w -= weight(p0[t]);
        }
        w = warp_sum(w);
        // to every CTA of the cluster. (Two sets: a CTA may be a pass ahead of one that
        // still reads, and not more.)
        if (lane < ctas) *cl.map_shared_rank(&sm.all[pass & 1][mine], lane) = w;
        cl.sync();
        unsigned long long z = 0;
        for (int i = lane; i < segs; i += 32) z += sm.all[pass & 1][i];
        ++pass;
        return warp_sum(z);
    };

    double z = 1.0;
    unsigned long long Z = 0;
    bool summed = false;                     // Z and sm.wsum are of R as it is
    for (int s = 1; s < n; ++s) {
        if (par[s] != cur) continue;
        const int x = tok[s];
        double rx;
        if (qb) {
            rx = static_cast<double>(rest(p0[s], q0[s]));
        } else {
            // rejected before: R(x) is 0 (every thread notes it, all the same)
            for (int t = cur + 1; t < s; ++t)
                if (par[t] == cur && tok[t] == x) p0[s] = 0.0f;
            __syncwarp();
            rx = static_cast<double>(p0[s]);
        }
        if (static_cast<double>(un[s]) * z * static_cast<double>(q0[s]) < rx) {
            if (rank == 0 && tid == 0) {
                path[acc] = s;
                tokens[acc - 1] = x;
            }
            ++acc;
            cur = s;
            rej = 0;
            summed = false;
            z = 1.0;
            prow = pb + static_cast<int64_t>(cur) * a.V;
            if (qb) qrow = qb + static_cast<int64_t>(cur) * a.V;
        } else if (qb) {
            if (rej == 0) zc = zc == zs ? zs + a.S1 : zs;
            zc[rej] = static_cast<float>(z);
            __syncwarp();
            ++rej;
            Z = sums(true);
            summed = true;
            z = static_cast<double>(static_cast<float>(static_cast<double>(Z) * 0x1p-45));
        } else {
            ++rej;
            z -= rx;
        }
    }
    // ---- the draw ----
    bool all_of_p = false;                   // R is empty: p takes its place
    if (!summed) Z = sums(false);
    if (Z == 0) {
        all_of_p = true;
        rej = 0;
        Z = sums(false);
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
        const unsigned long long* all = sm.all[(pass - 1) & 1];
        const float u0 = un[0];
        unsigned long long t = u0 > 0.0f ? static_cast<unsigned long long>(static_cast<double>(u0) * static_cast<double>(Z)) : 0ull;
        if (t >= Z) t = Z - 1;
        unsigned long long before = 0;
        for (int i = lane; i < mine; i += 32) before += all[i];
        before = warp_sum(before);
        if (t >= before && t - before < all[mine]) {
            auto weight_at = [&](int i) -> unsigned long long {
                const float r = __ldg(prow + i);
                return weight(qb && rej > 0 ? rest(r, __ldg(qrow + i)) : r);
            };
            // the weights of cur's rejected tokens in [from, to) (given drafts only)
            auto out = [&](int from, int to) {
                unsigned long long w = 0;
                for (int e = cur + 1; e < n && !qb && !all_of_p; ++e)
                    if (par[e] == cur && tok[e] >= from && tok[e] < to) w += weight(p0[e]);
                return w;
            };
            auto scan = [&](unsigned long long c) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned long long up = __shfl_up_sync(0xffffffffu, c, o);
                    if (lane >= o) c += up;
                }
                return c;
            };
            // the 32nd of the segment that holds it (one lane sums each), then the
            // value, 32 at a time
            const int sub = a.seg / 32, l0 = min(lo + lane * sub, hi), l1 = min(l0 + sub, hi);
            unsigned long long c = 0;
#pragma unroll 8
            for (int i = l0; i < l1; ++i) c += weight_at(i);
            c -= out(l0, l1);
            const unsigned long long upto = scan(c);
            const int at = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, before + upto > t))) - 1;
            before += __shfl_sync(0xffffffffu, upto - c, at);
            const int end = __shfl_sync(0xffffffffu, l1, at);
            for (int i0 = __shfl_sync(0xffffffffu, l0, at); i0 < end; i0 += 32) {
                const int i = i0 + lane;
                const unsigned long long v = scan(i < end ? weight_at(i) - out(i, i + 1) : 0ull);
                const unsigned hit = __ballot_sync(0xffffffffu, before + v > t);
                if (hit) {
                    if (lane == 0) tokens[acc - 1] = i0 + __ffs(static_cast<int>(hit)) - 1;
                    break;
                }
                before += __shfl_sync(0xffffffffu, v, 31);
            }
        }
    }
}

// ---- the accepted branch in the cache ------------------------------------------------
// One CTA per (sequence, heads_per_cta heads). A round takes rows in order as far
// as the CTA's registers go (kKBatch 16-byte chunks a thread): all are read, then,
// behind a barrier, written. path[i] >= i, so a round's writes, to lower rows
// than any later round's sources, spoil nothing that is still to be read.
// Latency-bound: a chain of four dependent loads (accepted, path, block table,
// row), which more rows do not lengthen.
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
    __shared__ int64_t src[kMaxNodes], dst[kMaxNodes];   // rows of head 0; src -1: no move
    const int b = blockIdx.x, tid = threadIdx.x;
    const int act = max(__ldg(p.act + b), 0);
    int n = p.len ? __ldg(p.len + b) : p.S1;
    n = n < 0 ? 0 : (n > p.S1 ? p.S1 : n);
    n = min(n, act);
    int m = __ldg(p.accepted + b);
    m = m < 0 ? 0 : (m > n ? n : m);
    const int ctx = act - n;
    if (blockIdx.y == 0 && tid == 0) p.new_act[b] = ctx + m;
    auto row0 = [&](int pos) -> int64_t {
        const int bi = pos / p.BS;
        if (pos < 0 || bi >= p.max_blocks) return -1;
        const int id = __ldg(p.bt + static_cast<int64_t>(b) * p.max_blocks + bi);
        return id >= 0 && id < p.num_blocks ? cache_row(p.layout, id, pos - bi * p.BS, 0, p.BS, p.H) : -1;
    };
    for (int i = tid; i < m; i += kKThreads) {
        const int s = __ldg(p.path + static_cast<int64_t>(b) * p.S1 + i);
        int64_t from = -1, to = -1;
        if (s != i && s >= 0 && s < n) {
            from = row0(ctx + s);
            to = row0(ctx + i);
        }
        src[i] = to >= 0 ? from : -1;
        dst[i] = to;
    }
    __syncthreads();
    const int64_t head_step = p.layout == PA_LAYOUT_BSND ? 1 : p.BS;
    const int h0 = blockIdx.y * p.heads_per_cta, heads = min(p.heads_per_cta, p.H - h0);
    const int per_row = heads * 2 * p.chunks;            // chunks of K, then of V, head by head
    const int rows = max(1, min(kKThreads * kKBatch / per_row, kKThreads / heads));   // a round's
    for (int i0 = 0; i0 < m; i0 += rows) {
        const int tasks = min(rows, m - i0) * per_row;
        uint4 v[kKBatch];
        uint4* to[kKBatch];
        float sv = 0.0f;
        float* sto = nullptr;
#pragma unroll
        for (int j = 0; j < kKBatch; ++j) {
            const int t = tid + j * kKThreads;
            to[j] = nullptr;
            if (t < tasks) {
                const int i = t / per_row, r = t - i * per_row;
                const int c = r / p.chunks, k = r - c * p.chunks;
                const int64_t from = src[i0 + i];
                if (from >= 0) {
                    const int64_t head = (h0 + (c >> 1)) * head_step;
                    uint4* base = reinterpret_cast<uint4*>((c & 1) ? p.vc : p.kc) + k;
                    v[j] = base[(from + head) * p.chunks];
                    to[j] = base + (dst[i0 + i] + head) * p.chunks;
                }
            }
        }
        if (tid < min(rows, m - i0) * heads) {
            const int i = tid / heads;
            if (src[i0 + i] >= 0) {
                const int64_t head = (h0 + tid - i * heads) * head_step;
                sv = p.ks[src[i0 + i] + head];
                sto = p.ks + dst[i0 + i] + head;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kKBatch; ++j)
            if (to[j]) *to[j] = v[j];
        if (sto) *sto = sv;
        __syncthreads();
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
    // (tensors of no sequences may have no address)
    PA_REQUIRE(B == 0 || (target_probs && draft_tokens && parents && uniforms && accepted && path && tokens),
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
    a.accepted = accepted;
    a.path = path;
    a.tokens = tokens;
    int cluster = kMaxCluster;
    while (cluster > 1 && static_cast<int64_t>(B) * cluster > kResident) cluster >>= 1;
    // segments of whole 128-value steps
    const int segs = cluster * kVWarps;
    a.seg = (V + segs * 128 - 1) / (segs * 128) * 128;
    const size_t smem = sizeof(VerifySmem) + static_cast<size_t>(S1) * 7 * sizeof(float);
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(B) * cluster);
    lc.blockDim = dim3(kVThreads);
    lc.dynamicSmemBytes = smem;
    lc.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    // rows that all start on 16 bytes are read 16 bytes at a time
    const bool vec = V % 4 == 0 && aligned(target_probs, 16) && aligned(draft_probs, 16);
    const cudaError_t e = vec ? cudaLaunchKernelEx(&lc, tree_verify_kernel<true>, a)
                              : cudaLaunchKernelEx(&lc, tree_verify_kernel<false>, a);
    PA_REQUIRE(e == cudaSuccess, PA_ERR_CUDA, "pa_tree_verify: launch: %s", cudaGetErrorString(e));
    return PA_OK;
}

extern "C" pa_status pa_fp8_cache_keep_path(void* key_cache, void* value_cache, float* key_scale_cache,
                                            const int32_t* block_table, const int32_t* kv_act_seqs,
                                            const int32_t* tree_len, const int32_t* path,
                                            const int32_t* accepted, int32_t* new_act_seqs, int B, int S1,
                                            int NKV, int head_size, int block_size, int64_t num_blocks,
                                            int max_blocks_per_seq, int layout, void* stream)
{
    const char* name = "pa_fp8_cache_keep_path";
    PA_REQUIRE(key_cache && value_cache && key_scale_cache &&
                   (B == 0 || (block_table && kv_act_seqs && path && accepted && new_act_seqs)),
               PA_ERR_NULLPTR, "%s: NULL tensor pointer", name);
    PA_REQUIRE(B >= 0 && S1 > 0 && NKV > 0 && head_size > 0 && block_size > 0 && num_blocks > 0 &&
                   max_blocks_per_seq > 0,
               PA_ERR_INVALID, "%s: empty or negative size", name);
    PA_REQUIRE(layout == PA_LAYOUT_BSND || layout == PA_LAYOUT_BNBD, PA_ERR_INVALID,
               "%s: unknown layout %d", name, layout);
    PA_REQUIRE(S1 <= kMaxNodes, PA_ERR_UNSUPPORTED, "%s: S1 %d > %d", name, S1, kMaxNodes);
    PA_REQUIRE(head_size % 16 == 0 && head_size <= 8192, PA_ERR_UNSUPPORTED,
               "%s: head_size %d (a multiple of 16 up to 8192)", name, head_size);
    static_assert(2 * 2 * 8192 / 16 <= kKThreads * kKBatch, "a row of two heads fits a round");
    PA_REQUIRE(B == 0 || new_act_seqs != kv_act_seqs, PA_ERR_INVALID,
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
    p.heads_per_cta = NKV < 2 ? 1 : 2;
    const int64_t gy = (NKV + p.heads_per_cta - 1) / p.heads_per_cta;
    PA_REQUIRE(gy <= 65535, PA_ERR_UNSUPPORTED, "%s: too many heads (%d)", name, NKV);
    cache_keep_path_kernel<<<dim3(static_cast<unsigned>(B), static_cast<unsigned>(gy)), kKThreads, 0,
                             static_cast<cudaStream_t>(stream)>>>(p);
    return check_launch(name);
}

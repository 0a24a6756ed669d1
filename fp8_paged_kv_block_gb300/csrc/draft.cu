// draft.cu -- verification of drafted tokens against the target's
// probabilities, and the accepted branch kept in the paged cache.
#include "common.cuh"

#include <cooperative_groups.h>

#include <algorithm>

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
// the w-th segment of the vocabulary, replays R there and sums it; for the draw
// the CTA with the segment that holds the value splits it between its warps.
// The weights are 2^-45 integers: their sums are exact, so the drawn index
// depends neither on the number of CTAs nor on the order of summation.
//
// Bound by the chain launch, gather (two loads), then per rejection a pass over
// the row and an exchange between the CTAs: about 1.5 us of start, 3 us a pass.
// 64 sequences of 16 nodes x 131072 values take 23 to 32 us by their random numbers
// (of 67 MB read once, 10 us at the copy rate; the sequence with the most has four
// passes), 256 of 5 x 50000 29 to 38 us, one of 8 x 32003 without probabilities 8 us.
// What made the chain short (on inputs of the 64 that take 27 us now):
// - code: a launch runs most of it once, and cold code comes from L2. With passes
//   and draw inlined and unrolled (61 KB a kernel instead of 27) the 64 took 39 us.
// - four 16-byte loads of p and of q in flight a lane: with two 39 us, and 512
//   threads a CTA, which wait longer for one another, 32.
// - FP64 tests only where FP32 cannot tell, see below.
// Sums pushed under mbarriers instead of a cluster barrier gained 1 us of 27 and
// were not kept.
//
// A sequence gets 8 CTAs while the batch's CTAs number at most kCtasPerSm an SM, half
// as many for twice the batch: more CTAs shorten a pass, and cost launches and
// exchanges. 4 or 8 an SM (one or two rounds of the GPU): 45 or 41 us on 128
// sequences of 16 x 131072, 60 or 53 on 500 of 5 x 50000, 29 or 30 on 256.
constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSegs = kMaxCluster * kVWarps;
constexpr int kMaxV = 1 << 18;
constexpr int kCtasPerSm = 8;

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
    const float x = fminf(fmaxf(r, 0.0f), 1.0f);
    const float t = __fmaf_rz(x, 0x1p22f, 0x1p23f);
    const float rest = __fmaf_rn(x, 0x1p22f, 0x1p23f - t);
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

// R after `rej` rejections of drawn drafts at four places, from p and q there
__device__ __forceinline__ void replay(float4& r, const float4& q, float z)
{
    r.x = fmaxf(__fsub_rn(r.x, __fmul_rn(z, q.x)), 0.0f);
    r.y = fmaxf(__fsub_rn(r.y, __fmul_rn(z, q.y)), 0.0f);
    r.z = fmaxf(__fsub_rn(r.z, __fmul_rn(z, q.z)), 0.0f);
    r.w = fmaxf(__fsub_rn(r.w, __fmul_rn(z, q.w)), 0.0f);
}

// Four values of a row in [lo, hi), zeros behind: STRIDE 1: i .. i + 3 (VEC: hi a
// multiple of 4), else i, i + STRIDE, ..
template <bool VEC, int STRIDE>
__device__ __forceinline__ float4 load4(const float* row, int i, int hi)
{
    if (VEC) return i < hi ? __ldg(reinterpret_cast<const float4*>(row + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(i < hi ? __ldg(row + i) : 0.0f, i + STRIDE < hi ? __ldg(row + i + STRIDE) : 0.0f,
                       i + 2 * STRIDE < hi ? __ldg(row + i + 2 * STRIDE) : 0.0f,
                       i + 3 * STRIDE < hi ? __ldg(row + i + 3 * STRIDE) : 0.0f);
}

// R's weights over [lo, hi), summed by a warp. One copy of it for all callers: a
// launch runs most of its code once, and what it fetches costs more than the call.
template <bool VEC>
__device__ __noinline__ unsigned long long weights_of(const float* prow, const float* qrow, const float* zs, int rej,
                                                      int lo, int hi)
{
    const int lane = threadIdx.x & 31;
    constexpr int kBatch = 4;                // 128-value steps whose loads are in flight at once
    unsigned long long w = 0;
#pragma unroll 1
    for (int i = lo; i < hi; i += 128 * kBatch) {
        float4 r[kBatch], q[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int at = i + 128 * j + (VEC ? 4 * lane : lane);
            r[j] = load4<VEC, 32>(prow, at, hi);
            if (rej > 0) q[j] = load4<VEC, 32>(qrow, at, hi);
        }
#pragma unroll 1
        for (int k = 0; k < rej; ++k) {
            const float z = zs[k];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) replay(r[j], q[j], z);
        }
        uint32_t h = 0, l = 0;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            add_weight(r[j].x, h, l);
            add_weight(r[j].y, h, l);
            add_weight(r[j].z, h, l);
            add_weight(r[j].w, h, l);
        }
        w += (static_cast<unsigned long long>(h - 4 * kBatch * kBias) << 23) + (l - 4 * kBatch * kBias);
    }
    return warp_sum(w);
}

struct VerifySmem {
    unsigned long long all[2][kMaxSegs];     // the cluster's segments' sums, by pass parity
    unsigned long long part[kVWarps];
    // then, S1 long each: p and q at a node's token, u, the z's (two sets), parent, token
};

template <bool VEC>
__global__ void __launch_bounds__(kVThreads, 4) tree_verify_kernel(const VerifyParams a)
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
#pragma unroll 1
            for (int i = tid; i < a.S1; i += kVThreads) path[i] = tokens[i] = -1;
            if (tid == 0) a.accepted[b] = 0;
        }
        return;
    }
    // (no CTA writes into another's shared memory before that one has started)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const float* pb = a.p + b * a.S1 * a.V;
    const float* qb = a.q ? a.q + b * a.S1 * a.V : nullptr;
#pragma unroll 1
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
    // current node, nodes accepted, drafts of cur rejected so far, where they end
    int cur = 0, acc = 1, rej = 0, last = 0;
    // The z's of cur's rejections. Every thread writes them, all the same, so that no
    // barrier is needed before they are read; a node's first takes the set that the
    // last node with rejections did not, as a slower warp may still be there (it has
    // passed that node's own cluster barrier, so no more than one set behind).
    float* zc = zs + a.S1;
    // R's weights in [from, to), summed by this warp: with drawn drafts p less z q for
    // each rejection, else p less the rejected drafts (a repeated one has p0 0)
    bool all_of_p = false;                   // R is empty: p takes its place
    auto part = [&](int from, int to) {
        unsigned long long w = weights_of<VEC>(prow, qrow, zc, qb ? rej : 0, from, to);
        if (!qb && !all_of_p)
#pragma unroll 1
            for (int t = cur + 1; t < last; ++t)
                if (par[t] == cur && tok[t] >= from && tok[t] < to) w -= weight(p0[t]);
        return w;
    };
    // R's weights summed over all of the vocabulary, and each segment's into sm.all
    int pass = 0;
    auto sums = [&] {
        const unsigned long long w = part(lo, hi);
        // to every CTA of the cluster. (Two sets: a CTA may be a pass ahead of one that
        // still reads, and not more.)
        if (lane < ctas) *cl.map_shared_rank(&sm.all[pass & 1][mine], lane) = w;
        cl.sync();
        unsigned long long z = 0;
#pragma unroll 1
        for (int i = lane; i < segs; i += 32) z += sm.all[pass & 1][i];
        ++pass;
        return warp_sum(z);
    };

    // z as FP32: exact with drawn drafts, within z_err of the FP64 value without
    float z = 1.0f, z_err = 0.0f;
    unsigned long long Z = 0;
    bool summed = false;                     // Z and sm.all are of R as it is
    int s = 1;
#pragma unroll 1
    for (;;) {
        // ---- to the next rejection of a drawn draft, or the end ----
        bool rejected = false;
#pragma unroll 1
        for (; s < n && !rejected; ++s) {
            if (par[s] != cur) continue;
            const int x = tok[s];
            float rx = p0[s];
            if (qb) {
#pragma unroll 1
                for (int k = 0; k < rej; ++k) rx = fmaxf(__fsub_rn(rx, __fmul_rn(zc[k], q0[s])), 0.0f);
            } else {
                // rejected before: R(x) is 0 (every thread notes it, all the same)
#pragma unroll 1
                for (int t = cur + 1; t < s; ++t)
                    if (par[t] == cur && tok[t] == x) p0[s] = 0.0f;
                __syncwarp();
                rx = p0[s];
            }
            // u z Q < R, in FP64 only where FP32 cannot tell: FP64 runs at two lanes a clock
            // and SM, and all of the cluster's warps do this (5 us of 45 on 64 sequences).
            // Three roundings of 2^-24 each are below 2^-20 of the product; what underflows
            // is below 2^-130 as long as Q <= 2^20.
            const float u = un[s], prod = u * z * q0[s], err = fabsf(prod) * 0x1p-20f + z_err * fabsf(u) + 0x1p-120f;
            bool take = prod + err < rx;
            if ((!take && !(prod - err > rx)) || !(fabsf(u) <= 1.0f && fabsf(q0[s]) <= 0x1p20f)) {
                double zd = z;
                if (!qb) {
                    zd = 1.0;
#pragma unroll 1
                    for (int t = cur + 1; t < s; ++t)
                        if (par[t] == cur) zd -= static_cast<double>(p0[t]);
                }
                take = static_cast<double>(u) * zd * static_cast<double>(q0[s]) < static_cast<double>(rx);
            }
            if (take) {
                if (rank == 0 && tid == 0) {
                    path[acc] = s;
                    tokens[acc - 1] = x;
                }
                ++acc;
                cur = s;
                rej = 0;
                last = 0;
                summed = false;
                z = 1.0f;
                z_err = 0.0f;
                prow = pb + static_cast<int64_t>(cur) * a.V;
                if (qb) qrow = qb + static_cast<int64_t>(cur) * a.V;
            } else if (qb) {
                if (rej == 0) zc = zc == zs ? zs + a.S1 : zs;
                zc[rej] = z;
                __syncwarp();
                ++rej;
                rejected = true;
            } else {
                last = s + 1;
                z -= rx;
                z_err += fabsf(z) * 0x1p-23f;
            }
        }
        if (rejected || !summed) Z = sums();
        summed = true;
        z = __ull2float_rn(Z) * 0x1p-45f;
        if (rejected) continue;
        if (Z != 0 || all_of_p) break;
        all_of_p = true;
        rej = 0;
        summed = false;
    }
    // ---- the draw ----
    if (rank == 0) {
        if (tid == 0) {
            a.accepted[b] = acc;
            path[0] = 0;
            if (Z == 0) tokens[acc - 1] = -1;
        }
#pragma unroll 1
        for (int i = acc + tid; i < a.S1; i += kVThreads) path[i] = tokens[i] = -1;
    }
    if (Z == 0) return;
    // The value lies where t = floor(u0 Z) does. Each CTA looks for it in its own
    // segments; the one that has it splits that segment between its warps.
    const unsigned long long* all = sm.all[(pass - 1) & 1];
    unsigned long long before = 0, here = 0;
#pragma unroll 1
    for (int i = lane; i < (rank + 1) * kVWarps; i += 32) (i < rank * kVWarps ? before : here) += all[i];
    before = warp_sum(before);
    here = warp_sum(here);
    // (FP64 again only where FP32 finds t in or near these segments)
    const float u0 = fminf(fmaxf(un[0], 0.0f), 1.0f);      // (NaN: 0)
    const float tf = u0 * __ull2float_rn(Z), near = tf * 0x1p-20f + 4.0f;
    if (__ull2float_rn(before) - near > tf || __ull2float_rn(before + here) + near < tf) return;
    unsigned long long t = static_cast<unsigned long long>(static_cast<double>(u0) * static_cast<double>(Z));
    if (t >= Z) t = Z - 1;
    if (t < before || t - before >= here) return;          // (the whole CTA, as above)
    int at = rank * kVWarps;
#pragma unroll 1
    while (t - before >= all[at]) before += all[at++];
    const int s0 = min(at * a.seg, a.V), s1 = min(s0 + a.seg, a.V);
    const int sub = (a.seg / 128 + kVWarps - 1) / kVWarps * 128;
    const int from = min(s0 + warp * sub, s1), to = min(from + sub, s1);
    const unsigned long long own = part(from, to);
    if (lane == 0) sm.part[warp] = own;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < warp; ++i) before += sm.part[i];
    if (t < before || t - before >= own) return;           // this warp has it
    const int k0 = qb ? rej : 0;
#pragma unroll 1
    for (int i0 = from; i0 < to; i0 += 128) {
        const int i = i0 + 4 * lane;
        float4 r = load4<VEC, 1>(prow, i, to);
        if (k0 > 0) {
            const float4 q = load4<VEC, 1>(qrow, i, to);
#pragma unroll 1
            for (int k = 0; k < k0; ++k) replay(r, q, zc[k]);
        }
        if (!qb && !all_of_p) {
#pragma unroll 1
            for (int e = cur + 1; e < last; ++e) {
                const int d = par[e] == cur ? tok[e] - i : -1;
                r.x = d == 0 ? 0.0f : r.x;
                r.y = d == 1 ? 0.0f : r.y;
                r.z = d == 2 ? 0.0f : r.z;
                r.w = d == 3 ? 0.0f : r.w;
            }
        }
        const unsigned long long w0 = weight(r.x), w1 = w0 + weight(r.y), w2 = w1 + weight(r.z), w3 = w2 + weight(r.w);
        unsigned long long v = w3;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long up = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + v > t);
        if (hit) {
            if (lane == __ffs(static_cast<int>(hit)) - 1) {
                const unsigned long long b = before + v - w3;
                tokens[acc - 1] = i + (b + w0 > t ? 0 : b + w1 > t ? 1 : b + w2 > t ? 2 : 3);
            }
            return;
        }
        before += __shfl_sync(0xffffffffu, v, 31);
    }
}

// ---- the accepted branch in the cache ------------------------------------------------
// One CTA per (sequence, heads_per_cta heads): four heads of 128 channels. A round takes rows in order as far
// as the CTA's registers go (kKBatch 16-byte chunks a thread): all are read, then,
// behind a barrier, written. path[i] >= i, so a round's writes, to lower rows
// than any later round's sources, spoil nothing that is still to be read.
// Latency-bound: a chain of three dependent loads (lengths and path, block table,
// row), which more rows do not lengthen: 4.1 us a pass on 16 sequences of 16 nodes x 8
// heads, 8.2 us on 256 of 64 (8.8 when 10.7 were taken with two heads a CTA, 8 chunks
// a thread and the divisions in the unrolled loop: 24 KB of code instead of 12, and
// 1024 CTAs of which 608 fit; 11.3 with eight heads a CTA, 12 with 8 chunks).
constexpr int kKThreads = 256;
constexpr int kKHeads = 4, kKBatch = 4, kKResident = 6;   // (6 CTAs an SM: 40 registers)

struct KeepParams {
    uint8_t *kc, *vc;
    float* ks;
    const int *bt, *act, *len, *path, *accepted;
    int* new_act;
    int S1, H, chunks, BS;
    int64_t num_blocks;
    int max_blocks, layout, heads_per_cta;
    uint32_t chunk_mul;                      // 2^20 / chunks + 1: r / chunks = r chunk_mul >> 20 while r chunks < 2^20
};

__global__ void __launch_bounds__(kKThreads, kKResident) cache_keep_path_kernel(const KeepParams p)
{
    __shared__ int64_t src[kMaxNodes], dst[kMaxNodes];   // rows of head 0; src -1: no move
    const int b = blockIdx.x, tid = threadIdx.x;
    const int* path = p.path + static_cast<int64_t>(b) * p.S1;
    int s = tid < p.S1 ? __ldg(path + tid) : -1;         // (with the loads below, not behind them)
    const int act = max(__ldg(p.act + b), 0);
    int n = p.len ? __ldg(p.len + b) : p.S1;
    int m = __ldg(p.accepted + b);
    n = min(n < 0 ? 0 : (n > p.S1 ? p.S1 : n), act);
    m = m < 0 ? 0 : (m > n ? n : m);
    const int ctx = act - n;
    if (blockIdx.y == 0 && tid == 0) p.new_act[b] = ctx + m;
    auto row0 = [&](int pos) -> int64_t {
        const int bi = pos / p.BS;
        if (pos < 0 || bi >= p.max_blocks) return -1;
        const int id = __ldg(p.bt + static_cast<int64_t>(b) * p.max_blocks + bi);
        return id >= 0 && id < p.num_blocks ? cache_row(p.layout, id, pos - bi * p.BS, 0, p.BS, p.H) : -1;
    };
#pragma unroll 1
    for (int i = tid; i < m; i += kKThreads) {
        if (i != tid) s = __ldg(path + i);
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
    // this thread's first chunk of a round (row i, chunk r of it), and its next ones' distance
    const int i_first = tid / per_row, r_first = tid - i_first * per_row;
    const int i_step = kKThreads / per_row, r_step = kKThreads - i_step * per_row;
#pragma unroll 1
    for (int i0 = 0; i0 < m; i0 += rows) {
        const int end = min(rows, m - i0);
        uint4 v[kKBatch];
        uint4* to[kKBatch];
        float sv = 0.0f;
        float* sto = nullptr;
        int i = i_first, r = r_first;
#pragma unroll
        for (int j = 0; j < kKBatch; ++j) {
            to[j] = nullptr;
            if (i < end && src[i0 + i] >= 0) {
                const int c = static_cast<int>(r * p.chunk_mul >> 20), k = r - c * p.chunks;
                const int64_t head = (h0 + (c >> 1)) * head_step;
                uint4* base = reinterpret_cast<uint4*>((c & 1) ? p.vc : p.kc) + k;
                v[j] = base[(src[i0 + i] + head) * p.chunks];
                to[j] = base + (dst[i0 + i] + head) * p.chunks;
            }
            i += i_step;
            r += r_step;
            if (r >= per_row) {
                r -= per_row;
                ++i;
            }
        }
        if (tid < end * heads) {
            const int si = tid / heads;
            if (src[i0 + si] >= 0) {
                const int64_t head = (h0 + tid - si * heads) * head_step;
                sv = p.ks[src[i0 + si] + head];
                sto = p.ks + dst[i0 + si] + head;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kKBatch; ++j)
            if (to[j]) *to[j] = v[j];
        if (sto) *sto = sv;
        if (i0 + rows < m) __syncthreads();
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
    // a sequence's CTAs read the inputs while one of them already writes
    const uint64_t rows = static_cast<uint64_t>(B) * S1, probs = rows * V * sizeof(float);
    const struct { const void* at; uint64_t bytes; } bufs[] = {
        {accepted, 4ull * B}, {path, 4 * rows}, {tokens, 4 * rows}, {target_probs, probs}, {draft_probs, probs},
        {draft_tokens, 4 * rows}, {parents, 4 * rows}, {uniforms, 4 * rows}, {tree_len, 4ull * B}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 9; ++j)
            PA_REQUIRE(!overlap(bufs[i].at, bufs[i].bytes, bufs[j].at, bufs[j].bytes), PA_ERR_INVALID,
                       "pa_tree_verify: accepted, path and tokens must overlap no other buffer");
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
    const int sms = device_sm_count();
    PA_REQUIRE(sms > 0, PA_ERR_CUDA, "pa_tree_verify: cannot query the device");
    while (cluster > 1 && static_cast<int64_t>(B) * cluster > kCtasPerSm * sms) cluster >>= 1;
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
    static_assert(2 * 8192 / 16 <= kKThreads * kKBatch, "a head's row fits a round");
    PA_REQUIRE(aligned(key_cache, 16) && aligned(value_cache, 16) && aligned(key_scale_cache, 4) &&
                   aligned(block_table, 4) && aligned(kv_act_seqs, 4) && aligned(tree_len, 4) && aligned(path, 4) &&
                   aligned(accepted, 4) && aligned(new_act_seqs, 4),
               PA_ERR_INVALID, "%s: misaligned pointer", name);
    if (B == 0) return PA_OK;
    // a sequence's CTAs read the inputs while one of them already writes
    const uint64_t ints = 4ull * B;
    PA_REQUIRE(!overlap(new_act_seqs, ints, kv_act_seqs, ints) && !overlap(new_act_seqs, ints, tree_len, ints) &&
                   !overlap(new_act_seqs, ints, accepted, ints) && !overlap(new_act_seqs, ints, path, ints * S1) &&
                   !overlap(new_act_seqs, ints, block_table, ints * max_blocks_per_seq),
               PA_ERR_INVALID, "%s: new_act_seqs must overlap no input (kv_act_seqs among them)", name);
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
    // a row of a CTA's heads fits a round
    p.heads_per_cta = std::min(NKV, std::max(1, std::min(kKHeads, kKThreads * kKBatch / (2 * p.chunks))));
    p.chunk_mul = (1u << 20) / p.chunks + 1;
    const int64_t gy = (NKV + p.heads_per_cta - 1) / p.heads_per_cta;
    PA_REQUIRE(gy <= 65535, PA_ERR_UNSUPPORTED, "%s: too many heads (%d)", name, NKV);
    cache_keep_path_kernel<<<dim3(static_cast<unsigned>(B), static_cast<unsigned>(gy)), kKThreads, 0,
                             static_cast<cudaStream_t>(stream)>>>(p);
    return check_launch(name);
}

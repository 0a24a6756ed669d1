// tree.cu -- attention of a tree of drafted tokens over the paged FP8 cache.
#include "common.cuh"

#include <cuda_fp8.h>

#include <cmath>

namespace pa {
namespace {

constexpr int kD = 128;
constexpr int kBS = 128;
constexpr int kMaxNodes = 128;
constexpr int kMaxGroup = 128;
constexpr int kMaxB = 1024;
constexpr size_t kWsHeader = 256;

struct TreeParams {
    const uint8_t* q;
    const float* q_scale;
    const uint8_t* kc;
    const float* k_scale;
    const uint8_t* vc;
    const float* v_scale;
    const int *bt, *act, *len;
    const uint8_t* mask;
    int64_t mask_stride;
    __nv_bfloat16* out;
    int S1, NQ, NKV;
    int64_t num_blocks;
    int max_blocks, layout;
    float scale_log2;
};

__device__ __forceinline__ float e4m3_to_float(uint8_t c)
{
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
}

// One CTA per query row (b, s, h): tiles of 128 keys, thread = key for the
// scores, thread = channel for the output; running maximum and sum.
__global__ void __launch_bounds__(kD) tree_decode_kernel(const TreeParams p)
{
    __shared__ float qf[kD], pr[kD], red[4];
    __shared__ int64_t rows[kD];
    const int tid = threadIdx.x, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const int h = static_cast<int>(row % p.NQ);
    const int64_t t = row / p.NQ;
    const int b = static_cast<int>(t / p.S1), s = static_cast<int>(t - static_cast<int64_t>(b) * p.S1);
    const int h2 = h / (p.NQ / p.NKV);
    const int act = max(min(static_cast<int64_t>(__ldg(p.act + b)), static_cast<int64_t>(p.max_blocks) * kBS), static_cast<int64_t>(0));
    int n = p.len ? __ldg(p.len + b) : p.S1;
    n = min(max(n, 0), min(p.S1, act));
    const int ctx = act - n;
    qf[tid] = e4m3_to_float(p.q[row * kD + tid]) * p.q_scale[row] * p.scale_log2;
    __syncthreads();
    float M = -INFINITY, L = 0.0f, o = 0.0f;
    if (s < n) {
        for (int j0 = 0; j0 < act; j0 += kD) {
            const int j = j0 + tid;
            bool see = j < act;
            if (see && j >= ctx) see = p.mask[b * p.mask_stride + static_cast<int64_t>(s) * p.S1 + (j - ctx)] != 0;
            float x = -INFINITY;
            int64_t r = 0;
            if (j < act) {
                int blk = __ldg(p.bt + static_cast<int64_t>(b) * p.max_blocks + j / kBS);
                if (blk < 0 || blk >= p.num_blocks) blk = 0;
                r = cache_row(p.layout, blk, j % kBS, h2, kBS, p.NKV);
            }
            if (see) {
                float d = 0.0f;
                for (int c = 0; c < kD; ++c) d += qf[c] * e4m3_to_float(p.kc[r * kD + c]);
                x = d * p.k_scale[r];
            }
            float m = warp_max_f32(x);
            if ((tid & 31) == 0) red[warp] = m;
            __syncthreads();
            m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
            const float Mn = fmaxf(M, m), ref = Mn == -INFINITY ? 0.0f : Mn;
            const float f = ex2(M - ref);
            pr[tid] = ex2(x - ref);
            rows[tid] = r;
            __syncthreads();
            M = Mn;
            L *= f;
            o *= f;
            const int lim = min(kD, act - j0);
            for (int k = 0; k < lim; ++k) {
                L += pr[k];
                o += pr[k] * e4m3_to_float(p.vc[rows[k] * kD + tid]);
            }
            __syncthreads();
        }
    }
    const float vs = p.v_scale[(static_cast<int64_t>(b) * p.NKV + h2) * kD + tid];
    p.out[row * kD + tid] = __float2bfloat16_rn(L > 0.0f ? o * vs / L : 0.0f);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pa_status check_shape(const char* name, int B, int S1, int NQ, int NKV, int D)
{
    PA_REQUIRE(B >= 0 && S1 > 0 && NQ > 0 && NKV > 0 && D > 0, PA_ERR_INVALID,
               "%s: negative or empty shape (B=%d S1=%d NQ=%d NKV=%d D=%d)", name, B, S1, NQ, NKV, D);
    PA_REQUIRE(NQ % NKV == 0, PA_ERR_INVALID, "%s: NQ %d is not a multiple of NKV %d", name, NQ, NKV);
    PA_REQUIRE(D == kD, PA_ERR_UNSUPPORTED, "%s: head size %d (only 128 is built)", name, D);
    PA_REQUIRE(B <= kMaxB, PA_ERR_UNSUPPORTED, "%s: batch %d > %d", name, B, kMaxB);
    PA_REQUIRE(S1 <= kMaxNodes, PA_ERR_UNSUPPORTED, "%s: S1 %d > %d drafted tokens", name, S1, kMaxNodes);
    PA_REQUIRE(NQ / NKV <= kMaxGroup, PA_ERR_UNSUPPORTED, "%s: %d query heads per kv head (at most %d)", name,
               NQ / NKV, kMaxGroup);
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_fp8_tree_decode_workspace_size(int B, int S1, int NQ, int NKV, int D, size_t* bytes)
{
    PA_REQUIRE(bytes, PA_ERR_NULLPTR, "pa_fp8_tree_decode_workspace_size: bytes is NULL");
    const pa_status st = check_shape("pa_fp8_tree_decode", B, S1, NQ, NKV, D);
    if (st != PA_OK) return st;
    *bytes = kWsHeader;
    return PA_OK;
}

extern "C" pa_status pa_fp8_tree_decode(const void* q, const float* q_scale, const void* k_cache,
                                        const float* k_scale, const void* v_cache, const float* v_scale,
                                        const int32_t* block_table, const int32_t* kv_act_seqs,
                                        const int32_t* tree_len, const uint8_t* tree_mask, int64_t mask_stride,
                                        void* out, int B, int S1, int NQ, int NKV, int D, int block_size,
                                        int64_t num_blocks, int max_blocks_per_seq, int layout,
                                        float softmax_scale, void* workspace, size_t workspace_bytes,
                                        void* stream)
{
    const char* name = "pa_fp8_tree_decode";
    PA_REQUIRE(q && q_scale && k_cache && k_scale && v_cache && v_scale && block_table && kv_act_seqs && tree_mask &&
                   out,
               PA_ERR_NULLPTR, "%s: NULL tensor pointer", name);
    size_t need = 0;
    const pa_status ps = pa_fp8_tree_decode_workspace_size(B, S1, NQ, NKV, D, &need);
    if (ps != PA_OK) return ps;
    PA_REQUIRE(num_blocks > 0 && max_blocks_per_seq > 0 && block_size > 0, PA_ERR_INVALID,
               "%s: empty cache or block table", name);
    PA_REQUIRE(block_size == kBS, PA_ERR_UNSUPPORTED, "%s: block_size %d (only 128 is built)", name, block_size);
    PA_REQUIRE(layout == PA_LAYOUT_BSND || layout == PA_LAYOUT_BNBD, PA_ERR_INVALID, "%s: unknown layout %d", name,
               layout);
    PA_REQUIRE(static_cast<int64_t>(max_blocks_per_seq) * kBS <= 0x7FFFFFFF, PA_ERR_UNSUPPORTED,
               "%s: block table wider than 2^31 - 1 positions", name);
    PA_REQUIRE(num_blocks * kBS * NKV <= 0x7FFFFFFF, PA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 cache rows", name);
    PA_REQUIRE(std::isfinite(softmax_scale), PA_ERR_INVALID, "%s: softmax_scale not finite", name);
    PA_REQUIRE(mask_stride >= 0, PA_ERR_INVALID, "%s: negative mask_stride", name);
    PA_REQUIRE(aligned16(q) && aligned16(k_cache) && aligned16(v_cache) && aligned16(v_scale) && aligned16(out),
               PA_ERR_INVALID, "%s: q, the caches, v_scale and out must be 16-byte aligned", name);
    if (B == 0) return PA_OK;
    PA_REQUIRE(workspace && workspace_bytes >= need, PA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name,
               workspace ? workspace_bytes : static_cast<size_t>(0), need);
    PA_REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, PA_ERR_INVALID,
               "%s: workspace must be 256-byte aligned", name);
    TreeParams p;
    p.q = static_cast<const uint8_t*>(q);
    p.q_scale = q_scale;
    p.kc = static_cast<const uint8_t*>(k_cache);
    p.k_scale = k_scale;
    p.vc = static_cast<const uint8_t*>(v_cache);
    p.v_scale = v_scale;
    p.bt = block_table;
    p.act = kv_act_seqs;
    p.len = tree_len;
    p.mask = tree_mask;
    p.mask_stride = mask_stride;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.S1 = S1;
    p.NQ = NQ;
    p.NKV = NKV;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.layout = layout;
    p.scale_log2 = softmax_scale * 1.4426950408889634f;
    tree_decode_kernel<<<static_cast<unsigned>(B) * S1 * NQ, kD, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return check_launch(name);
}

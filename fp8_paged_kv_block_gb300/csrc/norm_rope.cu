// norm_rope.cu -- per-head RMSNorm and rotation of q and k, E4M3 quantisation,
// and the append of k and v to the paged cache, in one pass.
//
// A row is one head of one token: y = x * rsqrt(mean(x^2) + eps) * w, the
// first rotary_dim channels rotated in pairs by the position's angles, scale =
// max|y| / 448, codes E4M3(y * (448 / max|y|)). One read of each input value
// and one write of each code: bound by those bytes on long prompts, by the
// launch and one chain of dependent loads on a few tokens.
//
// A row's head_size values lie 8 to a lane, so that a BF16 row is one 16-byte
// load per lane: 16 lanes per row of 128, two rows to a warp, and the sums and
// maxima take four shuffles for both. A warp takes kSets of those, heads of one
// token and of one kind (q, k or v), with all loads in flight at once: angles and
// weights stay in registers over them. (A job of rows numbered straight through,
// with a 64-bit division and its own angles for every row, took 188 us on the
// 8192-token case.)
#include "common.cuh"

#include <cmath>

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kSets = 4;

struct NormRopeParams {
    const void *q, *k, *v;
    int64_t qs, ks, vs;               // elements from one token to the next
    const void *qw, *kw;
    int w_bf16;
    float eps;
    const float* cos_sin;
    int rd;
    int64_t max_pos;
    const void* pos;
    int pos_type;
    uint8_t* q_codes;
    float* q_scale;
    uint8_t *kc, *vc;
    const void* slots;
    int slot_type;
    float* k_scale;
    const float* v_scale;
    const int* token_batch;
    int num_batches;
    int64_t T;
    int NQ, NKV;
    uint32_t q_jobs, kv_jobs;                // warps a token's q heads, its k (and v) heads take
    int64_t num_blocks;
    int BS, layout;
};

__device__ __forceinline__ void unpack_bf16(uint4 v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8])
{
    unpack_bf16(__ldg(reinterpret_cast<const uint4*>(p)), x);
}

// Eight values as they lie in memory, unpacked where they are used.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const
    {
        x[0] = make_float2(a.x, a.y); x[1] = make_float2(a.z, a.w);
        x[2] = make_float2(b.x, b.y); x[3] = make_float2(b.z, b.w);
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
};

// Eight codes of y * (448 / amax). Where the quotient may leave the float range
// both sides are first taken times a power of two.
__device__ __forceinline__ uint2 encode8(float2 (&y)[4], float amax)
{
    if (!(amax >= 0x1p-100f && amax <= 0x1p100f)) {
        if (amax == 0.0f) return make_uint2(0u, 0u);
        const float up = amax < 1.0f ? 0x1p100f : 0x1p-100f;
        amax *= up;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __fmul2_rn(y[e], make_float2(up, up));
    }
    const float inv = __fdividef(kE4M3Max, amax);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __fmul2_rn(y[e], make_float2(inv, inv));
    return make_uint2(e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y), e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y));
}

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 6) qkv_norm_rope_append_kernel(const NormRopeParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = kSets * RPW;
    const int lane = threadIdx.x & 31, sub = lane % LPR, d0 = 8 * sub;
    const uint32_t job = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t per_token = p.q_jobs + 2 * p.kv_jobs;
    const uint32_t tok = job / per_token;
    if (tok >= p.T) return;
    uint32_t part = job - tok * per_token;
    const bool is_q = part < p.q_jobs, is_v = part >= p.q_jobs + p.kv_jobs;
    if (!is_q) part -= is_v ? p.q_jobs + p.kv_jobs : p.q_jobs;
    const int heads = is_q ? p.NQ : p.NKV;
    const int h0 = static_cast<int>(part) * ROWS + lane / LPR;
    const T* src = is_q ? static_cast<const T*>(p.q) + tok * p.qs
                   : is_v ? static_cast<const T*>(p.v) + tok * p.vs
                          : static_cast<const T*>(p.k) + tok * p.ks;

    // (the angles wait for the position: it goes first)
    int64_t pos = p.rd > 0 && !is_v ? load_slot(p.pos, p.pos_type, tok) : 0;
    Raw8<T> raw[kSets];
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
        const int h = h0 + i * RPW;
        if (h < heads) raw[i].load(src + h * D + d0);
        else raw[i].zero();
    }
    // where k and v go
    int64_t row = -1, row_step = 0;          // cache row of head 0, from head to head
    if (!is_q) {
        const int64_t s = load_slot(p.slots, p.slot_type, tok);
        if (s < 0 || s >= p.num_blocks * p.BS) return;
        const int64_t blk = s / p.BS, off = s - blk * p.BS;
        row = cache_row(p.layout, blk, off, 0, p.BS, p.NKV);
        row_step = p.layout == PA_LAYOUT_BSND ? 1 : p.BS;
    }
    if (is_v) {
        int tb = __ldg(p.token_batch + tok);
        tb = tb < 0 ? 0 : (tb >= p.num_batches ? p.num_batches - 1 : tb);
        const float* vs = p.v_scale + static_cast<int64_t>(tb) * p.NKV * D + d0;
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            const int h = h0 + i * RPW;
            if (h >= heads) break;
            float2 x[4];
            float sc[8], z[8];
            raw[i].get(x);
            load8(vs + h * D, sc);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[e] = sc[e] == 0.0f ? 0.0f : __fdiv_rn((e & 1) ? x[e >> 1].y : x[e >> 1].x, sc[e]);
            uint2 c;
            c.x = e4m3x4(z[0], z[1], z[2], z[3]);
            c.y = e4m3x4(z[4], z[5], z[6], z[7]);
            *reinterpret_cast<uint2*>(p.vc + (row + h * row_step) * D + d0) = c;
        }
        return;
    }
    // ---- this lane's weights and angles ----
    const void* w = is_q ? p.qw : p.kw;
    float2 wt[4];
    {
        float t[8];
        if (w == nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = 1.0f;
        } else if (p.w_bf16) {
            load8(static_cast<const __nv_bfloat16*>(w) + d0, t);
        } else {
            load8(static_cast<const float*>(w) + d0, t);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) wt[e] = make_float2(t[2 * e], t[2 * e + 1]);
    }
    const int half = p.rd >> 1;
    const bool rot = d0 < p.rd, low = d0 < half;
    // channel i's partner sits rd / 16 lanes up or down (INTER: in the same lane)
    const int from = lane + (!INTER && rot ? (low ? half >> 3 : -(half >> 3)) : 0);
    float2 cs[4], sn[4];                     // per channel (INTER: a pair's in both)
    if (rot) {
        pos = pos < 0 ? 0 : (pos >= p.max_pos ? p.max_pos - 1 : pos);
        const float* a = p.cos_sin + pos * p.rd;
        if constexpr (INTER) {
            const float4 c4 = __ldg(reinterpret_cast<const float4*>(a + (d0 >> 1)));
            const float4 s4 = __ldg(reinterpret_cast<const float4*>(a + half + (d0 >> 1)));
            cs[0] = make_float2(c4.x, c4.x); cs[1] = make_float2(c4.y, c4.y);
            cs[2] = make_float2(c4.z, c4.z); cs[3] = make_float2(c4.w, c4.w);
            sn[0] = make_float2(-s4.x, s4.x); sn[1] = make_float2(-s4.y, s4.y);
            sn[2] = make_float2(-s4.z, s4.z); sn[3] = make_float2(-s4.w, s4.w);
        } else {
            float t[8];
            load8(a + (low ? d0 : d0 - half), t);
#pragma unroll
            for (int e = 0; e < 4; ++e) cs[e] = make_float2(t[2 * e], t[2 * e + 1]);
            load8(a + half + (low ? d0 : d0 - half), t);
            const float sign = low ? -1.0f : 1.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sn[e] = make_float2(sign * t[2 * e], sign * t[2 * e + 1]);
        }
    }
    // this lane's 8 codes of head h0, and from one set to the next
    uint8_t* dst = is_q ? p.q_codes + (static_cast<int64_t>(tok) * p.NQ + h0) * D + d0
                        : p.kc + (row + h0 * row_step) * D + d0;
    const int64_t dst_step = (is_q ? RPW : RPW * row_step) * D;
    float mine = 0.0f;                       // max|y| of the row whose scale this lane writes
#pragma unroll
    for (int i = 0; i < kSets; ++i, dst += dst_step) {
        // every lane takes part in the shuffles, whatever its row is
        float2 y[4];
        raw[i].get(y);
        if (w != nullptr) {
            float2 s2 = __fmul2_rn(y[0], y[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) s2 = __ffma2_rn(y[e], y[e], s2);
            float ss = s2.x + s2.y, sc = 1.0f;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            // squares that leave the float range (or, with no eps to speak of, vanish
            // below it) are taken of x * 2^-64 (2^64)
            const bool big = !(ss <= 1e38f), small = ss < 1e-30f && p.eps < 1e-20f;
            if (__any_sync(0xffffffffu, big || small)) {
                sc = big ? 0x1p-64f : (small ? 0x1p64f : 1.0f);
                ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 t = __fmul2_rn(y[e], make_float2(sc, sc));
                    ss += t.x * t.x + t.y * t.y;
                }
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            }
            const float ms = ss * (1.0f / D) + p.eps * sc * sc;
            const float inv = ms == 0.0f ? 0.0f : rsqrtf(ms) * sc;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = __fmul2_rn(__fmul2_rn(y[e], make_float2(inv, inv)), wt[e]);
        }
        if (INTER || p.rd > 0) {
            float2 o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (INTER) {
                    o[e] = make_float2(y[e].y, y[e].x);
                } else {
                    o[e].x = __shfl_sync(0xffffffffu, y[e].x, from);
                    o[e].y = __shfl_sync(0xffffffffu, y[e].y, from);
                }
            }
            if (rot) {
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = __ffma2_rn(o[e], sn[e], __fmul2_rn(y[e], cs[e]));
            }
        }
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(fmaxf(amax, fabsf(y[e].x)), fabsf(y[e].y));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        mine = sub == i ? amax : mine;
        if (h0 + i * RPW < heads) *reinterpret_cast<uint2*>(dst) = encode8(y, amax);
    }
    // the scales of all rows at once: lane i of a row's lanes has set i's
    const int h = h0 + sub * RPW;
    if (sub < kSets && h < heads)
        (is_q ? p.q_scale + static_cast<int64_t>(tok) * p.NQ + h : p.k_scale + row + h * row_step)[0] =
            __fdiv_rn(mine, kE4M3Max);
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename T, int D>
void launch(NormRopeParams p, bool inter, cudaStream_t st)
{
    constexpr uint32_t rows = kSets * (32 / (D / 8));        // rows a warp takes
    p.q_jobs = (p.NQ + rows - 1) / rows;
    p.kv_jobs = (p.NKV + rows - 1) / rows;
    constexpr int warps = kThreads / 32;
    const unsigned grid = static_cast<unsigned>((p.T * (p.q_jobs + 2 * p.kv_jobs) + warps - 1) / warps);
    if (inter) qkv_norm_rope_append_kernel<T, D, true><<<grid, kThreads, 0, st>>>(p);
    else qkv_norm_rope_append_kernel<T, D, false><<<grid, kThreads, 0, st>>>(p);
}

template <typename T>
void launch_d(const NormRopeParams& p, int D, bool inter, cudaStream_t st)
{
    if (D == 64) launch<T, 64>(p, inter, st);
    else if (D == 128) launch<T, 128>(p, inter, st);
    else launch<T, 256>(p, inter, st);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_fp8_qkv_norm_rope_append(
    const void* q, const void* k, const void* v, int in_dtype, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, const void* q_weight, const void* k_weight, int weight_dtype, float eps,
    const float* cos_sin, int rotary_dim, int64_t max_position, int interleaved,
    const void* positions, int pos_type, void* q_codes, float* q_scale, void* key_cache,
    void* value_cache, const void* slot_mapping, int slot_type, float* key_scale_cache,
    const float* v_scale, const int32_t* token_batch, int num_batches, int64_t num_tokens, int NQ,
    int NKV, int head_size, int64_t num_blocks, int block_size, int layout, void* stream)
{
    const char* name = "pa_fp8_qkv_norm_rope_append";
    // (tensors of no tokens may have no address)
    PA_REQUIRE(key_cache && value_cache && key_scale_cache && v_scale &&
                   (num_tokens == 0 || (q && k && v && q_codes && q_scale && slot_mapping && token_batch)),
               PA_ERR_NULLPTR, "%s: NULL tensor pointer", name);
    PA_REQUIRE(num_tokens >= 0 && NQ > 0 && NKV > 0 && head_size > 0 && num_blocks > 0 &&
                   block_size > 0 && num_batches > 0,
               PA_ERR_INVALID, "%s: empty or negative size", name);
    PA_REQUIRE(head_size == 64 || head_size == 128 || head_size == 256, PA_ERR_UNSUPPORTED,
               "%s: head_size %d (64, 128 and 256 are built)", name, head_size);
    PA_REQUIRE(rotary_dim >= 0 && rotary_dim <= head_size, PA_ERR_INVALID,
               "%s: rotary_dim %d outside [0, head_size]", name, rotary_dim);
    PA_REQUIRE(rotary_dim % (interleaved ? 8 : 16) == 0, PA_ERR_UNSUPPORTED,
               "%s: rotary_dim %d (a multiple of 16, or of 8 if interleaved)", name, rotary_dim);
    PA_REQUIRE(rotary_dim == 0 || (cos_sin && (positions || num_tokens == 0)), PA_ERR_NULLPTR,
               "%s: NULL cos_sin or positions", name);
    PA_REQUIRE(rotary_dim == 0 || max_position > 0, PA_ERR_INVALID, "%s: empty cos_sin", name);
    PA_REQUIRE(in_dtype == PA_DTYPE_F32 || in_dtype == PA_DTYPE_BF16, PA_ERR_INVALID,
               "%s: unknown input dtype %d", name, in_dtype);
    PA_REQUIRE(weight_dtype == PA_DTYPE_F32 || weight_dtype == PA_DTYPE_BF16, PA_ERR_INVALID,
               "%s: unknown weight dtype %d", name, weight_dtype);
    PA_REQUIRE((slot_type == PA_INDEX_I32 || slot_type == PA_INDEX_I64) &&
                   (pos_type == PA_INDEX_I32 || pos_type == PA_INDEX_I64),
               PA_ERR_INVALID, "%s: unknown slot or position type", name);
    PA_REQUIRE(layout == PA_LAYOUT_BSND || layout == PA_LAYOUT_BNBD, PA_ERR_INVALID,
               "%s: unknown layout %d", name, layout);
    PA_REQUIRE(std::isfinite(eps) && eps >= 0.0f, PA_ERR_INVALID, "%s: eps is negative or not finite", name);
    const int64_t per16 = in_dtype == PA_DTYPE_F32 ? 4 : 8;
    PA_REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && q_stride % per16 == 0 &&
                   k_stride % per16 == 0 && v_stride % per16 == 0,
               PA_ERR_INVALID, "%s: q, k and v tokens must start on 16-byte boundaries", name);
    PA_REQUIRE(aligned(q_weight, 16) && aligned(k_weight, 16) && aligned(cos_sin, 16) &&
                   aligned(v_scale, 16) && aligned(q_codes, 8) && aligned(key_cache, 8) &&
                   aligned(value_cache, 8) && aligned(q_scale, 4) && aligned(key_scale_cache, 4),
               PA_ERR_INVALID, "%s: misaligned pointer", name);
    PA_REQUIRE(num_tokens <= 0x7FFFFFFF && num_tokens * (static_cast<int64_t>(NQ) + 2 * NKV) < (static_cast<int64_t>(1) << 32),
               PA_ERR_UNSUPPORTED, "%s: more than 2^32 head rows", name);
    if (num_tokens == 0) return PA_OK;
    NormRopeParams p;
    p.q = q; p.k = k; p.v = v;
    p.qs = q_stride; p.ks = k_stride; p.vs = v_stride;
    p.qw = q_weight; p.kw = k_weight;
    p.w_bf16 = weight_dtype == PA_DTYPE_BF16;
    p.eps = eps;
    p.cos_sin = cos_sin;
    p.rd = rotary_dim;
    p.max_pos = max_position;
    p.pos = positions;
    p.pos_type = pos_type;
    p.q_codes = static_cast<uint8_t*>(q_codes);
    p.q_scale = q_scale;
    p.kc = static_cast<uint8_t*>(key_cache);
    p.vc = static_cast<uint8_t*>(value_cache);
    p.slots = slot_mapping;
    p.slot_type = slot_type;
    p.k_scale = key_scale_cache;
    p.v_scale = v_scale;
    p.token_batch = token_batch;
    p.num_batches = num_batches;
    p.T = num_tokens;
    p.NQ = NQ;
    p.NKV = NKV;
    p.num_blocks = num_blocks;
    p.BS = block_size;
    p.layout = layout;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (in_dtype == PA_DTYPE_F32) launch_d<float>(p, head_size, interleaved != 0, st);
    else launch_d<__nv_bfloat16>(p, head_size, interleaved != 0, st);
    return check_launch(name);
}

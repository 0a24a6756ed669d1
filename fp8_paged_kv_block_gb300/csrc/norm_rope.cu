// norm_rope.cu -- per-head RMSNorm and rotation of q and k, E4M3 quantisation,
// and the append of k and v to the paged cache, in one pass.
//
// A row is one head of one token: y = x * rsqrt(mean(x^2) + eps) * w, the
// first rotary_dim channels rotated in pairs by the position's angles, scale =
// max|y| / 448, codes E4M3(y * (448 / max|y|)). One read of each input value
// and one write of each code: bound by those bytes on long prompts, by the
// launch and one chain of dependent loads on a few tokens.
//
// A row's head_size values lie 8 to a lane in two chunks of 4 channels: the two
// of a rotary lane hold the two sides of its four pairs, so that the rotation
// needs no other lane. A job is kSets sets of rows (two rows of 128 a set), heads
// of one token and of one kind (q, k or v). The sets' sums and maxima are reduced
// together, half of the sets to either lane at each of the first two steps, after
// which a lane has one set's and does that set's scalar work; 1 / rms is left out
// of the codes, which it cancels from, and goes into the scale alone.
//
// A warp takes a run of jobs, so that angles and weights last for a token's, and
// has the next job's rows on their way to shared memory while it works on one.
// 8192 tokens of 96 + 2 x 8 heads of 128: BF16 82 us a pass (358 MB of inputs and
// outputs, 4.4 TB/s; the instructions issue at 63% of the clocks, 560 a job of 8
// rows), FP32 95 us (593 MB, 6.2 TB/s). With a job a warp and its rows in registers
// BF16 took 107 us, FP32 115; rotating through shuffles and reducing each set by
// itself (820 instructions) 113 and 137. Three or four jobs in flight change nothing
// (83, 84); six CTAs an SM, at 80 registers with spills, 93. Few tokens: 16 take 4.1
// us one after another in a graph, 8 to 11 launched by the host; 777 of 48 + 2 x 8
// heads in FP32 8.6 us, 10 to 13.
#include "common.cuh"

#include <algorithm>
#include <cmath>

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kSets = 4;
constexpr int kBlocks = 5;                   // CTAs an SM: 96 registers
constexpr int kStages = 2;                   // jobs of a warp in shared memory
constexpr int kJob = kSets * 256;            // values of a job's rows

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
    uint32_t q_jobs, kv_jobs;                // jobs a token's q heads, its k (and v) heads make
    uint32_t per, longer;                    // jobs a warp, warps with one more
    int64_t num_blocks;
    int BS, layout;
};

// Four values as they lie in memory, unpacked where they are used.
__device__ __forceinline__ float4 load_raw(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ uint2 load_raw(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }
__device__ __forceinline__ float4 load_smem(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ uint2 load_smem(const __nv_bfloat16* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ void unpack(const float4& r, float2& a, float2& b)
{
    a = make_float2(r.x, r.y);
    b = make_float2(r.z, r.w);
}
__device__ __forceinline__ void unpack(const uint2& r, float2& a, float2& b)
{
    a = make_float2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u));
    b = make_float2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u));
}
__device__ __forceinline__ void prefetch_l1(const void* p, int type, uint32_t i)
{
    const char* at = static_cast<const char*>(p) + static_cast<int64_t>(i) * (type == PA_INDEX_I64 ? 8 : 4);
    asm volatile("prefetch.global.L1 [%0];" ::"l"(at));
}

// The larger one, NaN if either is: a NaN or what infinities make of one must not
// get lost in a row's maximum, as it would in fmaxf.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float2 times(float2 a, float f) { return __fmul2_rn(a, make_float2(f, f)); }

// One copy of the four divisions for all callers: only a few warps come here.
__device__ __noinline__ uint32_t value_codes(float2 a, float2 b, float4 s)
{
    return e4m3x4(s.x == 0.0f ? 0.0f : __fdiv_rn(a.x, s.x), s.y == 0.0f ? 0.0f : __fdiv_rn(a.y, s.y),
                  s.z == 0.0f ? 0.0f : __fdiv_rn(b.x, s.z), s.w == 0.0f ? 0.0f : __fdiv_rn(b.y, s.w));
}

// kSets values of a lane reduced over the `lpr` lanes of its row, set 2 (lane & 1)
// + (lane >> 1 & 1) to this lane.
template <bool MAX>
__device__ __forceinline__ float reduce_sets(const float (&a)[kSets], int lane, int lpr)
{
    static_assert(kSets == 4, "two steps halve the sets to one");
    auto op = [](float x, float y) { return MAX ? max_nan(x, y) : x + y; };
    const bool b0 = lane & 1, b1 = lane & 2;
    const float k0 = op(b0 ? a[2] : a[0], __shfl_xor_sync(0xffffffffu, b0 ? a[0] : a[2], 1));
    const float k1 = op(b0 ? a[3] : a[1], __shfl_xor_sync(0xffffffffu, b0 ? a[1] : a[3], 1));
    float v = op(b1 ? k1 : k0, __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2));
#pragma unroll
    for (int o = 4; o < lpr; o <<= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocks) qkv_norm_rope_append_kernel(const NormRopeParams p)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = kSets * RPW;
    __shared__ __align__(16) T ring[kThreads / 32][kStages][kJob];
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const uint32_t wid = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    T(*const mine)[kJob] = ring[threadIdx.x >> 5];
    // this warp's jobs
    const uint32_t begin = wid * p.per + min(wid, p.longer), end = begin + p.per + (wid < p.longer ? 1 : 0);
    if (begin == end) return;
    const uint32_t per_token = p.q_jobs + 2 * p.kv_jobs;

    // ---- rows on their way to shared memory, kStages - 1 jobs ahead ----
    uint32_t ahead = begin, a_tok = begin / per_token, a_part = begin - a_tok * per_token;
    int a_slot = 0;
    // the first token's position and slot on their way to L1 (the angles and rows wait
    // for them, and the rows' addresses take a while)
    if (p.rd > 0) prefetch_l1(p.pos, p.pos_type, a_tok);
    prefetch_l1(p.slots, p.slot_type, a_tok);
    auto fetch = [&] {
        if (ahead < end) {
            const bool q = a_part < p.q_jobs, v = a_part >= p.q_jobs + p.kv_jobs;
            const uint32_t part = q ? a_part : a_part - p.q_jobs - (v ? p.kv_jobs : 0);
            const T* src = (q ? static_cast<const T*>(p.q) + a_tok * p.qs
                            : v ? static_cast<const T*>(p.v) + a_tok * p.vs
                                : static_cast<const T*>(p.k) + a_tok * p.ks) + part * (ROWS * D);
            const int left = ((q ? p.NQ : p.NKV) - static_cast<int>(part) * ROWS) * D;   // values; zeros behind
#pragma unroll
            for (int i = 0; i < kJob * static_cast<int>(sizeof(T)) / 512; ++i) {
                const int at = (32 * i + lane) * (16 / static_cast<int>(sizeof(T)));
                cp_async16(mine[a_slot] + at, src + (at < left ? at : 0), at < left ? 16 : 0);
            }
            if (++a_part == per_token) {
                a_part = 0;
                ++a_tok;
            }
            ++ahead;
            a_slot = a_slot + 1 == kStages ? 0 : a_slot + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint32_t tok = a_tok, part_all = a_part;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();

    int slot_now = 0;
    bool fresh = true;                       // another token or kind than before
    int64_t row = -1, row_step = 0;          // k, v: cache row of head 0, from head to head
    int c0 = 0, c1 = 0;                      // this lane's chunks of 4 channels
    bool rot0 = false, rot1 = false;
    float2 wt[4], cs[2] = {}, sn[2] = {};    // its weights, the angles of its four pairs
#pragma unroll 1
    for (uint32_t job = begin; job < end; ++job) {
        const bool is_q = part_all < p.q_jobs, is_v = part_all >= p.q_jobs + p.kv_jobs;
        const uint32_t part = is_q ? part_all : part_all - p.q_jobs - (is_v ? p.kv_jobs : 0);
        const uint32_t t_now = tok;
        const T* const x = mine[slot_now];
        const int heads = is_q ? p.NQ : p.NKV;
        const int h0 = static_cast<int>(part) * ROWS + lane / LPR;
        const void* w = is_q ? p.qw : p.kw;
        if (fresh || part == 0) {
            const int rd = is_v ? 0 : p.rd, half = rd >> 1;
            int64_t pos = rd > 0 ? load_slot(p.pos, p.pos_type, t_now) : 0;
            const int64_t s = is_q ? 0 : load_slot(p.slots, p.slot_type, t_now);
            if (INTER) {
                c0 = 4 * sub;
                c1 = c0 + D / 2;
            } else {
                const bool in = 8 * sub < rd;
                c0 = in ? 4 * sub : rd + 4 * (sub - (rd >> 3));
                c1 = c0 + (in ? half : (D - rd) >> 1);
            }
            rot0 = c0 < rd;
            rot1 = INTER ? c1 < rd : rot0;
            if (!is_v) {
                if (w == nullptr) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) wt[e] = make_float2(1.0f, 1.0f);
                } else if (p.w_bf16) {
                    unpack(load_raw(static_cast<const __nv_bfloat16*>(w) + c0), wt[0], wt[1]);
                    unpack(load_raw(static_cast<const __nv_bfloat16*>(w) + c1), wt[2], wt[3]);
                } else {
                    unpack(load_raw(static_cast<const float*>(w) + c0), wt[0], wt[1]);
                    unpack(load_raw(static_cast<const float*>(w) + c1), wt[2], wt[3]);
                }
            }
            pos = pos < 0 ? 0 : (pos >= p.max_pos ? p.max_pos - 1 : pos);
            const float* a = p.cos_sin + pos * rd;
            if (INTER) {
                if (rot0) {
                    cs[0] = __ldg(reinterpret_cast<const float2*>(a + (c0 >> 1)));
                    sn[0] = __ldg(reinterpret_cast<const float2*>(a + half + (c0 >> 1)));
                }
                if (rot1) {
                    cs[1] = __ldg(reinterpret_cast<const float2*>(a + (c1 >> 1)));
                    sn[1] = __ldg(reinterpret_cast<const float2*>(a + half + (c1 >> 1)));
                }
            } else if (rot0) {
                unpack(load_raw(a + c0), cs[0], cs[1]);
                unpack(load_raw(a + half + c0), sn[0], sn[1]);
            }
            row = -1;
            row_step = p.layout == PA_LAYOUT_BSND ? 1 : p.BS;
            if (!is_q && s >= 0 && s < p.num_blocks * p.BS) {
                const int64_t blk = s >> 31 ? s / p.BS : static_cast<uint32_t>(s) / static_cast<uint32_t>(p.BS);
                row = cache_row(p.layout, blk, s - blk * p.BS, 0, p.BS, p.NKV);
            }
            fresh = false;
        }
        // the next job
        if (++part_all == per_token) {
            part_all = 0;
            ++tok;
            fresh = true;
        }
        slot_now = slot_now + 1 == kStages ? 0 : slot_now + 1;
        // (this warp is done with the slot that is filled now)
        __syncwarp();
        fetch();
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        if (!is_q && row < 0) continue;          // no slot
        const T* const lane_x = x + (lane / LPR) * D;
        if (is_v) {
            int tb = __ldg(p.token_batch + t_now);
            tb = tb < 0 ? 0 : (tb >= p.num_batches ? p.num_batches - 1 : tb);
            const float* vs = p.v_scale + static_cast<int64_t>(tb) * p.NKV * D;
            float4 sc[kSets][2];
#pragma unroll
            for (int i = 0; i < kSets; ++i) {
                const int h = min(h0 + i * RPW, heads - 1);
                sc[i][0] = load_raw(vs + h * D + c0);
                sc[i][1] = load_raw(vs + h * D + c1);
            }
#pragma unroll
            for (int i = 0; i < kSets; ++i) {
                const int h = h0 + i * RPW;
                if (h >= heads) break;
                uint8_t* out = p.vc + (row + h * row_step) * D;
                float2 a, b;
                unpack(load_smem(lane_x + i * RPW * D + c0), a, b);
                *reinterpret_cast<uint32_t*>(out + c0) = value_codes(a, b, sc[i][0]);
                unpack(load_smem(lane_x + i * RPW * D + c1), a, b);
                *reinterpret_cast<uint32_t*>(out + c1) = value_codes(a, b, sc[i][1]);
            }
            continue;
        }
        auto rotate = [&](float2 (&y)[4]) {
            if (INTER) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (e < 2 ? rot0 : rot1) {
                        const float c = (e & 1) ? cs[e >> 1].y : cs[e >> 1].x;
                        const float n = (e & 1) ? sn[e >> 1].y : sn[e >> 1].x;
                        y[e] = make_float2(y[e].x * c - y[e].y * n, y[e].y * c + y[e].x * n);
                    }
                }
            } else if (rot0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 a = y[e], b = y[e + 2];
                    y[e] = __ffma2_rn(b, make_float2(-sn[e].x, -sn[e].y), __fmul2_rn(a, cs[e]));
                    y[e + 2] = __ffma2_rn(a, sn[e], __fmul2_rn(b, cs[e]));
                }
            }
        };
        auto max_of = [](const float2 (&y)[4]) {
            float m = max_nan(fabsf(y[0].x), fabsf(y[0].y));
#pragma unroll
            for (int e = 1; e < 4; ++e) m = max_nan(max_nan(m, fabsf(y[e].x)), fabsf(y[e].y));
            return m;
        };
        const int64_t q0 = static_cast<int64_t>(t_now) * p.NQ + h0;
        uint8_t* dst = is_q ? p.q_codes + q0 * D : p.kc + (row + h0 * row_step) * D;
        const int64_t dst_step = (is_q ? RPW : RPW * row_step) * D;
        float* const scale = is_q ? p.q_scale + q0 : p.k_scale + row + h0 * row_step;
        const int64_t scale_step = is_q ? RPW : RPW * row_step;
        // ---- z = x w, rotated; the sets' sums of x^2 and maxima of |z| ----
        float2 z[kSets][4];
        float ss[kSets], amax[kSets];
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            float2 (&y)[4] = z[i];
            unpack(load_smem(lane_x + i * RPW * D + c0), y[0], y[1]);
            unpack(load_smem(lane_x + i * RPW * D + c1), y[2], y[3]);
            float2 s2 = __fmul2_rn(y[0], y[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) s2 = __ffma2_rn(y[e], y[e], s2);
            ss[i] = s2.x + s2.y;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = __fmul2_rn(y[e], wt[e]);
            rotate(y);
            amax[i] = max_of(y);
        }
        const int own = 2 * (lane & 1) + (lane >> 1 & 1);        // the set this lane reduces
        const float ss_own = reduce_sets<false>(ss, lane, LPR), amax_own = reduce_sets<true>(amax, lane, LPR);
        // Squares, products or quotients out of the comfortable range, a row of zeros or one
        // with a NaN among them: done again below.
        const bool fine = (w == nullptr || (ss_own <= 1e38f && ss_own >= 1e-30f)) && amax_own >= 0x1p-100f &&
                          amax_own <= 0x1p100f;
        const int own_lane = lane - sub;                        // + (i >> 1) + 2 (i & 1): the lane with set i's
        // ---- codes z (448 / max|z|), and the scales ----
        const float f_own = __fdividef(kE4M3Max, amax_own);
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            const float f = __shfl_sync(0xffffffffu, f_own, own_lane + (i >> 1) + 2 * (i & 1));
#pragma unroll
            for (int e = 0; e < 4; ++e) z[i][e] = times(z[i][e], f);
            if (h0 + i * RPW < heads) {
                uint8_t* const at = dst + i * dst_step;
                *reinterpret_cast<uint32_t*>(at + c0) = e4m3x4(z[i][0].x, z[i][0].y, z[i][1].x, z[i][1].y);
                *reinterpret_cast<uint32_t*>(at + c1) = e4m3x4(z[i][2].x, z[i][2].y, z[i][3].x, z[i][3].y);
            }
        }
        const float s = __fdiv_rn(amax_own, kE4M3Max);
        if (sub < kSets && h0 + own * RPW < heads && fine)
            scale[own * scale_step] = w == nullptr ? s : s * rsqrtf(ss_own * (1.0f / D) + p.eps);
        // The other rows, one by one in the order that keeps all in range. (Only they: a
        // row's result does not depend on those beside it.) A row with a NaN, its own or an
        // infinity's, has the maximum NaN and so NaN codes and scale.
        if (__any_sync(0xffffffffu, !fine && h0 + own * RPW < heads)) {
#pragma unroll 1
            for (int i = 0; i < kSets; ++i, dst += dst_step) {
                const bool in = !__shfl_sync(0xffffffffu, fine, own_lane + (i >> 1) + 2 * (i & 1)) && h0 + i * RPW < heads;
                float2 y[4];
                unpack(load_smem(lane_x + i * RPW * D + c0), y[0], y[1]);
                unpack(load_smem(lane_x + i * RPW * D + c1), y[2], y[3]);
                float rms = 1.0f;
                if (w != nullptr) {
                    // times 2^64 or 2^-80 where squares would leave the range, then normalised
                    float t = max_of(y);
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, o));
                    const float f = t > 0x1p56f ? 0x1p-80f : (t < 0x1p-60f ? 0x1p64f : 1.0f);
                    t = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = times(y[e], f);
                        t += y[e].x * y[e].x + y[e].y * y[e].y;
                    }
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                    // (under an eps of 1e-20 and more, squares below 2^-120 do not count; the
                    // power of two then goes into the scale)
                    const bool eps_alone = f > 1.0f && p.eps >= 1e-20f;
                    const float ms = eps_alone ? p.eps : t * (1.0f / D) + p.eps * f * f;
                    const float inv = ms == 0.0f ? 0.0f : rsqrtf(ms);
                    rms = eps_alone ? 0x1p-64f : 1.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = __fmul2_rn(times(y[e], inv), wt[e]);
                }
                rotate(y);
                float m = max_of(y);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float up = m < 0x1p-100f ? 0x1p100f : (m > 0x1p100f ? 0x1p-100f : 1.0f);
                const float f = m == 0.0f ? 0.0f : __fdividef(kE4M3Max, m * up);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = times(times(y[e], up), f);
                if (!in) continue;
                *reinterpret_cast<uint32_t*>(dst + c0) = m == 0.0f ? 0u : e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y);
                *reinterpret_cast<uint32_t*>(dst + c1) = m == 0.0f ? 0u : e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y);
                if (sub == 0) scale[i * scale_step] = __fdiv_rn(m, kE4M3Max) * rms;
            }
        }
    }
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename T, int D>
void launch(NormRopeParams p, bool inter, int sms, cudaStream_t st)
{
    constexpr uint32_t rows = kSets * (32 / (D / 8));        // rows a warp takes
    p.q_jobs = (p.NQ + rows - 1) / rows;
    p.kv_jobs = (p.NKV + rows - 1) / rows;
    const uint32_t jobs = static_cast<uint32_t>(p.T) * (p.q_jobs + 2 * p.kv_jobs);
    constexpr uint32_t warps = kThreads / 32;
    const uint32_t ctas = std::min((jobs - 1) / warps + 1, static_cast<uint32_t>(sms * kBlocks));
    p.per = jobs / (ctas * warps);
    p.longer = jobs % (ctas * warps);
    if (inter) qkv_norm_rope_append_kernel<T, D, true><<<ctas, kThreads, 0, st>>>(p);
    else qkv_norm_rope_append_kernel<T, D, false><<<ctas, kThreads, 0, st>>>(p);
}

template <typename T>
void launch_d(const NormRopeParams& p, int D, bool inter, int sms, cudaStream_t st)
{
    if (D == 64) launch<T, 64>(p, inter, sms, st);
    else if (D == 128) launch<T, 128>(p, inter, sms, st);
    else launch<T, 256>(p, inter, sms, st);
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
                   aligned(value_cache, 8) && aligned(q_scale, 4) && aligned(key_scale_cache, 4) &&
                   aligned(token_batch, 4) && aligned(positions, pos_type == PA_INDEX_I64 ? 8 : 4) &&
                   aligned(slot_mapping, slot_type == PA_INDEX_I64 ? 8 : 4),
               PA_ERR_INVALID, "%s: misaligned pointer", name);
    PA_REQUIRE(num_tokens <= 0x7FFFFFFF && num_tokens * (static_cast<int64_t>(NQ) + 2 * NKV) < (static_cast<int64_t>(1) << 32),
               PA_ERR_UNSUPPORTED, "%s: more than 2^32 head rows", name);
    PA_REQUIRE(NQ <= 0x7FFFFFFF / head_size && NKV <= 0x7FFFFFFF / head_size, PA_ERR_UNSUPPORTED,
               "%s: a token of 2^31 values or more", name);
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
    const int sms = device_sm_count();
    PA_REQUIRE(sms > 0, PA_ERR_CUDA, "%s: cannot query the device", name);
    if (in_dtype == PA_DTYPE_F32) launch_d<float>(p, head_size, interleaved != 0, sms, st);
    else launch_d<__nv_bfloat16>(p, head_size, interleaved != 0, sms, st);
    return check_launch(name);
}

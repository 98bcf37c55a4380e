// rope.cu -- rotary positions, and per-head RMS norms of queries and keys with
// the rotation in the same pass (forward and backward).
//
// Mathematics.  Pair i of a head at position p turns by the angle
// a = 2 pi p t_i, where t_i is the pair's frequency in turns per position:
//   (x1, x2) -> m (x1 cos a - x2 sin a, x2 cos a + x1 sin a),
// and the gradient turns back by the same angle (the transpose).  The table
// holds t_i as a 64-bit fixed-point fraction, so p * t_i modulo one turn is
// exactly the low 64 bits of an integer product, at any position: a far
// position loses no bits to a large angle.  Its top 32 bits are the angle the
// kernels take the sine and cosine of, in fp32: off by 2^-25 of half a turn at
// most, 2^-14 of a bf16 rounding.  For fp32 tensors the nearest quarter turn is
// split off as an integer first, which leaves 2^-27 (the error of rotated rows
// falls from 6.1e-8 to 4.8e-8 of their norm; one per cent of the gradient
// kernel's time with 16-bit types, where it would be lost).
// With the norm, y = R(x r w) with r = 1 / sqrt(mean(x^2) + eps); backward
// (g = R^T dy, gw = g w):  dx = r (gw - x r^2 mean(gw x)),  dw = sum g x r.
// Everything between the load and the store is fp32; values are rounded once.
//
// Layout of the work.  A thread holds whole pairs, so no element crosses
// threads for the rotation and a row's sums are a shuffle over the L lanes
// that share the head.  A warp takes one token and walks passes of 32 / L
// heads; the sines and cosines of a token are computed once, by the warp
// together, for all of its query and key heads.
//   16-byte groups: eight pairs per thread, two 16-byte accesses (for 16-bit
//     types) per tensor; needs 16-byte aligned rows and D a multiple of 16.
//   single pairs: any even D and R, any strides; one head per pass.
// What bounds it: HBM, each element read and written once.  65536 tokens of 32/8
// heads, D = 128, bf16, rotated: 192 us, 7.0 TB/s; 32760 tokens of 24/24 heads
// normed and rotated: 126 us, 6.4 TB/s.  A few tokens: the launch.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "api_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace ctxattn {
namespace {

constexpr int kMaxRopeDim = 512;
constexpr int kWarps = 2;      // warps of a forward block
constexpr int kGradWarps = 4;  // warps of a norm-gradient block
// Of them on an SM: 16-bit types at 128 registers; fp32 and the shifted pairs,
// which hold twice the words or angles, at 168 (fp32 at 128 spills: 183 us
// instead of 125 on 10000 tokens of 24/24 heads, D = 128).
constexpr int kGradBlocks = 4, kGradBlocksWide = 3;
constexpr int kJoinedPasses = 4;  // up to which a rotation joins queries' and keys' heads (launch_rope_mode)
constexpr int kMaxGradBlocks = 1024;  // blocks of the backward that leave partial weight gradients

enum { kRotate = 0, kNorm = 1, kNormGrad = 2 };
// How a thread's sixteen elements of a row form pairs (16-byte groups below).
enum { kHalf = 0, kInter = 1, kShifted = 2 };

struct RopeRows {  // one logical [B,S,H,D] tensor
    const void* p;
    int64_t sb, ss, sh;
};

struct RopeParams {
    RopeRows x[2], g[2], y[2];  // q, k: input, incoming gradient (backward), result
    const void* w[2];           // norm weights [D], or null
    int H[2];                   // heads (0: tensor absent)
    int passes[2];              // passes of 32 / L heads
    int w_type;                 // ctx_dtype_t of the weights
    int B, S, D, rot, L, log2_L;
    int per_unit;               // passes of one unit of work (a warp's share of a token)
    int units_per_token;
    const uint64_t* turns;      // [rot / 2]
    const int64_t* pos;         // null: offset + s
    int64_t pos_sb, pos_ss, pos_sa, offset;
    int n_axes, sec_end[4];     // pairs [sec_end[a-1], sec_end[a]) use axis a
    int interleaved;
    int joined;                 // passes run over the queries' heads and then the keys' (passes[1] is 0)
    float m, sin_sign, eps;
    float* dw_part;             // [blocks][2][D], or null (a side without a tensor is not written)
    float* dw[2];
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float weight_at(const RopeParams& p, int side, int i) {
    if (!p.w[side]) return 1.f;
    return p.w_type == CTX_DTYPE_FP32 ? static_cast<const float*>(p.w[side])[i]
         : p.w_type == CTX_DTYPE_FP16 ? __half2float(static_cast<const __half*>(p.w[side])[i])
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(p.w[side])[i]);
}
template <typename T>
__device__ __forceinline__ T* token_row(const RopeRows& r, int b, int s) {
    return (T*)r.p + b * r.sb + s * r.ss;
}

// A warp's share of the work: one token (b, s) and a range of head passes.
struct Unit {
    int b, s, part;
};
// A token's rows by head: one side's, or the queries' and then the keys'.
template <typename T, bool kJoined>
struct HeadRows {
    T* row[kJoined ? 2 : 1];
    int64_t sh[kJoined ? 2 : 1];
    int first_k;
    __device__ __forceinline__ HeadRows(const RopeParams& p, const RopeRows* r, int side, const Unit& u) {
        first_k = p.H[0];
#pragma unroll
        for (int i = 0; i < (kJoined ? 2 : 1); ++i) {
            row[i] = token_row<T>(r[side + i], u.b, u.s);
            sh[i] = r[side + i].sh;
        }
    }
    __device__ __forceinline__ T* at(int h) const {
        return !kJoined || h < first_k ? row[0] + h * sh[0] : row[kJoined] + (h - first_k) * sh[kJoined];
    }
};
__device__ __forceinline__ Unit unit_at(const RopeParams& p, int64_t u) {
    const int64_t token = u / p.units_per_token;
    Unit r;
    r.part = (int)(u - token * p.units_per_token);
    r.b = (int)(token / p.S);
    r.s = (int)(token - (int64_t)r.b * p.S);
    return r;
}

// Where pair i's (cosine, sine) lies in the warp's table, in float2.  With
// 16-byte groups a thread reads two pairs per access; the threads of a row
// then read consecutive ones, so no two of them meet in a bank.
template <bool kVec>
__device__ __forceinline__ int angle_slot(int i, int ngroups) {
    return kVec ? (((i & 7) >> 1) * ngroups + (i >> 3)) * 2 + (i & 1) : i;
}

// The cosines and sines of one token, computed by the whole warp (each angle
// once, not once per head) and shared through `cs`.
template <bool kVec, bool kFine>
__device__ __forceinline__ void token_angles(const RopeParams& p, const Unit& u, float2* cs) {
    __syncwarp();  // the previous token's are no longer read
    for (int i = lane_id(); i < p.D / 2; i += 32) {
        float2 v = make_float2(1.f, 0.f);  // the part that is not rotated
        if (i < p.rot / 2) {
            int axis = 0;
            for (int a = 0; a + 1 < p.n_axes; ++a) axis += i >= p.sec_end[a];
            const int64_t at = p.pos ? p.pos[u.b * p.pos_sb + u.s * p.pos_ss + axis * p.pos_sa] : p.offset + u.s;
            const uint32_t turn = (uint32_t)(((uint64_t)at * p.turns[i]) >> 32);
            const uint32_t quarter = kFine ? (turn + (1u << 29)) >> 30 : 0;
            float si, co;
            sincospif((float)(int32_t)(turn - (quarter << 30)) * 4.656612873077393e-10f, &si, &co);  // 2^-31: half turns
            if constexpr (kFine) {
                const float s0 = si, c0 = co;
                si = (quarter & 1) ? c0 : s0;
                co = (quarter & 1) ? s0 : c0;
                if (quarter & 2) si = -si;
                if ((quarter + 1) & 2) co = -co;
            }
            v = make_float2(co * p.m, si * p.sin_sign);
        }
        cs[angle_slot<kVec>(i, p.D / 16)] = v;
    }
    __syncwarp();
}

// ------------------------------------------------------- 16-byte groups
// A thread's 16 elements of a row, as stored: eight neighbouring twos.
//   kInter    two j is pair j.
//   kHalf     twos 0..3 are the first elements of pairs 0..7, twos 4..7 their
//             second ones (R a multiple of 16).
//   kShifted  the half layout for any other R: sixteen consecutive elements,
//             whose partners, R / 2 away, other threads hold; they come through
//             shared memory (Partners).
template <typename T>
struct Group {
    uint4 u[sizeof(T)];  // 16 elements
    __device__ __forceinline__ void load(const T* row, int2 at) {
        constexpr int n = sizeof(T) / 2;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            u[i] = reinterpret_cast<const uint4*>(row + at.x)[i];
            u[n + i] = reinterpret_cast<const uint4*>(row + at.y)[i];
        }
    }
    __device__ __forceinline__ void store(T* row, int2 at) const {
        constexpr int n = sizeof(T) / 2;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            reinterpret_cast<uint4*>(row + at.x)[i] = u[i];
            reinterpret_cast<uint4*>(row + at.y)[i] = u[n + i];
        }
    }
    __device__ __forceinline__ uint32_t& word(int i) { return reinterpret_cast<uint32_t*>(u)[i]; }
    __device__ __forceinline__ uint32_t word(int i) const { return reinterpret_cast<const uint32_t*>(u)[i]; }
    __device__ __forceinline__ float2 two(int j) const {
        if constexpr (sizeof(T) == 4) {
            return make_float2(__uint_as_float(word(2 * j)), __uint_as_float(word(2 * j + 1)));
        } else if constexpr (std::is_same<T, __half>::value) {
            const uint32_t w = word(j);
            return __half22float2(*reinterpret_cast<const __half2*>(&w));
        } else {
            return make_float2(__uint_as_float(word(j) << 16), __uint_as_float(word(j) & 0xffff0000u));
        }
    }
    __device__ __forceinline__ float2 swapped(int j) const {
        const float2 v = two(j);
        return make_float2(v.y, v.x);
    }
    __device__ __forceinline__ void set(int j, float2 v) {
        if constexpr (sizeof(T) == 4) {
            word(2 * j) = __float_as_uint(v.x);
            word(2 * j + 1) = __float_as_uint(v.y);
        } else if constexpr (std::is_same<T, __half>::value) {
            const __half2 h = __floats2half2_rn(v.x, v.y);
            word(j) = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            word(j) = pack_bf16x2(v.x, v.y);
        }
    }
};

// The warp's rows in shared memory, word w of every lane side by side: writing
// a thread's own words and reading its partners' (all the same distance away)
// are both free of bank conflicts.
template <typename T>
struct Partners {
    static constexpr int kWords = 4 * sizeof(T);  // of a lane
    uint32_t* buf;
    __device__ __forceinline__ void put(const Group<T>& g) const {
        __syncwarp();  // the previous row's are no longer read
#pragma unroll
        for (int i = 0; i < kWords; ++i) buf[i * 32 + lane_id()] = g.word(i);
        __syncwarp();
    }
    // element e (of the row of this thread's head)
    __device__ __forceinline__ float at(int e, int row_lane0) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(buf[(e & 15) * 32 + row_lane0 + (e >> 4)]);
        } else {
            const int w = e >> 1;
            const T* two = reinterpret_cast<const T*>(buf + (w & 7) * 32 + row_lane0 + (w >> 3));
            return to_f<T>(two[e & 1]);
        }
    }
    // The partners of elements e, e + 1 (e even): R / 2 further, or back; an
    // element past R is its own (its sine is zero).
    __device__ __forceinline__ float2 pair(const RopeParams& p, int e, int row_lane0) const {
        const int h = p.rot / 2;
        const int e0 = e < h ? e + h : (e < p.rot ? e - h : e);
        if (sizeof(T) == 2 && (h & 1) == 0) {
            const int w = e0 >> 1;
            Group<T> g;
            g.word(0) = buf[(w & 7) * 32 + row_lane0 + (w >> 3)];
            return g.two(0);
        }
        const int f = e + 1, e1 = f < h ? f + h : (f < p.rot ? f - h : f);
        return make_float2(at(e0, row_lane0), at(e1, row_lane0));
    }
};

struct RowThread {  // which part of which head's row a thread holds
    int group, slot;
    int lane0;  // first lane of this head's row
    bool live;
    int2 at;  // where its two runs of eight elements start
    __device__ __forceinline__ RowThread(const RopeParams& p, int style) {
        const int lane = lane_id();
        slot = lane >> p.log2_L;
        group = lane & (p.L - 1);
        lane0 = lane - group;
        live = group < p.D / 16;
        if (!live) group = 0;  // reads the first group's elements; kept out of sums and stores
        at = style == kHalf && group * 8 < p.rot / 2 ? make_int2(group * 8, p.rot / 2 + group * 8)
                                             : make_int2(group * 16, group * 16 + 8);
    }
    // Sums over the row's lanes of N values at once (their shuffles overlap).
    template <int N>
    __device__ __forceinline__ void row_sums(const RopeParams& p, float (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (!live) v[i] = 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            if (o < p.L) {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
            }
    }
    // (cosine, sine) of pairs 2j, 2j + 1
    __device__ __forceinline__ float4 angles(const RopeParams& p, const float2* cs, int j) const {
        return *reinterpret_cast<const float4*>(cs + angle_slot<true>(group * 8 + 2 * j, p.D / 16));
    }
    // kShifted: (cosine, sine) of the pair element e belongs to, the sine with
    // the sign its partner enters with
    __device__ __forceinline__ float2 angle_of(const RopeParams& p, const float2* cs, int e) const {
        const int h = p.rot / 2;
        if (e >= p.rot) return make_float2(1.f, 0.f);
        const float2 v = cs[angle_slot<true>(e < h ? e : e - h, p.D / 16)];
        return make_float2(v.x, e < h ? -v.y : v.y);
    }
    __device__ __forceinline__ void weights(const RopeParams& p, int side, float2* w) const {
        if (!p.w[side]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = make_float2(1.f, 1.f);
        } else if (p.w_type == CTX_DTYPE_FP32) {
            Group<float> g;
            g.load(static_cast<const float*>(p.w[side]), at);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = g.two(j);
        } else if (p.w_type == CTX_DTYPE_FP16) {
            Group<__half> g;
            g.load(static_cast<const __half*>(p.w[side]), at);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = g.two(j);
        } else {
            Group<__nv_bfloat16> g;
            g.load(static_cast<const __nv_bfloat16*>(p.w[side]), at);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = g.two(j);
        }
    }
};

template <typename T>
__device__ __forceinline__ float row_rsqrt(float v) {
    // 2 ulp (2^-22) is far below half a step of a 16-bit type
    if constexpr (sizeof(T) == 4) return __frsqrt_rn(v);
    else return rsqrtf(v);
}

// Rotation (with the norm when kNormed): one unit per warp.  Everything that a
// token's heads share is folded into sixteen coefficients per thread, so that
// an element costs two products and the row's factor:
//   interleaved  y = x (wa c, wb c) + swap(x) (-wb s, wa s)
//   half         ya = a (wa c) + b (-wb s),  yb = b (wb c) + a (wa s)
// in two-lane fp32 instructions.  kBatch passes are loaded before the first
// is computed, so that a warp has kBatch kilobytes (16-bit types) in flight.
template <typename T, int kStyle, bool kNormed, bool kJoined, int kBatch, int kBlocks>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float2 cs_all[kWarps][kMaxRopeDim / 2];
    __shared__ uint32_t partners[kStyle == kShifted ? kWarps : 1][kStyle == kShifted ? 32 * Partners<T>::kWords : 1];
    const Partners<T> pt{partners[kStyle == kShifted ? warp_id() : 0]};
    float2* cs = cs_all[warp_id()];
    const int64_t un = (int64_t)blockIdx.x * kWarps + warp_id();
    if (un >= (int64_t)p.B * p.S * p.units_per_token) return;
    const RowThread th(p, kStyle);
    const int per_pass = 32 >> p.log2_L;
    const float inv_d = 1.f / (float)p.D;
    const Unit u = unit_at(p, un);
    const int first = u.part * p.per_unit, last = min(first + p.per_unit, p.passes[0] + p.passes[1]);
    bool have_angles = false;
    // both sides in line where registers allow: their strides and pointers are
    // then constants of the launch, not indexed loads (133 -> 126 us, below)
#pragma unroll(kNormed && kBatch > 2 ? 2 : 1)
    for (int side = 0; side < (kJoined ? 1 : 2); ++side) {
        const int base = side ? p.passes[0] : 0;
        const int p0 = max(first - base, 0), p1 = min(last - base, p.passes[side]);
        if (p0 >= p1) continue;
        const int H = kJoined ? p.H[0] + p.H[1] : p.H[side];
        const HeadRows<T, kJoined> xt(p, p.x, side, u), yt(p, p.y, side, u);
        float2 k[16];
        bool have_k = false;
#pragma unroll 1
        for (int ps = p0; ps < p1; ps += kBatch) {
            Group<T> raw[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (ps + i < p1) raw[i].load(xt.at(min((ps + i) * per_pass + th.slot, H - 1)), th.at);
            if (!have_angles) {
                token_angles<true, sizeof(T) == 4>(p, u, cs);
                have_angles = true;
            }
            if (!have_k) {
                float2 w[8];
                if constexpr (kNormed) th.weights(p, side, w);
#pragma unroll
                for (int j = 0; kStyle != kShifted && j < 4; ++j) {
                    const float4 a = th.angles(p, cs, j);  // pairs 2j, 2j + 1
                    if constexpr (kStyle == kInter) {
                        const float2 w0 = kNormed ? w[2 * j] : make_float2(1.f, 1.f);
                        const float2 w1 = kNormed ? w[2 * j + 1] : make_float2(1.f, 1.f);
                        k[2 * j] = make_float2(w0.x * a.x, w0.y * a.x);
                        k[2 * j + 1] = make_float2(w1.x * a.z, w1.y * a.z);
                        k[8 + 2 * j] = make_float2(-w0.y * a.y, w0.x * a.y);
                        k[8 + 2 * j + 1] = make_float2(-w1.y * a.w, w1.x * a.w);
                    } else {
                        const float2 wa = kNormed ? w[j] : make_float2(1.f, 1.f);
                        const float2 wb = kNormed ? w[4 + j] : make_float2(1.f, 1.f);
                        k[j] = make_float2(wa.x * a.x, wa.y * a.z);
                        k[4 + j] = make_float2(wb.x * a.x, wb.y * a.z);
                        k[8 + j] = make_float2(-wb.x * a.y, -wb.y * a.w);
                        k[12 + j] = make_float2(wa.x * a.y, wa.y * a.w);
                    }
                }
                if constexpr (kStyle == kShifted) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = th.group * 16 + 2 * j, hf = p.rot / 2;
                        const float2 a0 = th.angle_of(p, cs, e), a1 = th.angle_of(p, cs, e + 1);
                        float2 wo = make_float2(1.f, 1.f), wp = wo;  // own weights, partners' weights
                        if constexpr (kNormed) {
                            wo = w[j];
                            wp.x = weight_at(p, side, e < hf ? e + hf : (e < p.rot ? e - hf : e));
                            wp.y = weight_at(p, side, e + 1 < hf ? e + 1 + hf : (e + 1 < p.rot ? e + 1 - hf : e + 1));
                        }
                        k[j] = make_float2(wo.x * a0.x, wo.y * a1.x);
                        k[8 + j] = make_float2(wp.x * a0.y, wp.y * a1.y);
                    }
                }
                have_k = true;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (ps + i >= p1) continue;
                const int h = (ps + i) * per_pass + th.slot;
                float2 r2 = make_float2(1.f, 1.f);
                if constexpr (kNormed) {
                    float2 q = make_float2(0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) q = ffma2(raw[i].two(j), raw[i].two(j), q);
                    float sum[1] = {q.x + q.y};
                    th.row_sums(p, sum);
                    const float r = row_rsqrt<T>(fmaf(sum[0], inv_d, p.eps));
                    r2 = make_float2(r, r);
                }
                Group<T> y;
                if constexpr (kStyle == kShifted) pt.put(raw[i]);
                if constexpr (kStyle != kHalf) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 other = kStyle == kInter ? raw[i].swapped(j) : pt.pair(p, th.group * 16 + 2 * j, th.lane0);
                        float2 v = ffma2(raw[i].two(j), k[j], fmul2(other, k[8 + j]));
                        if constexpr (kNormed) v = fmul2(v, r2);
                        y.set(j, v);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 a = raw[i].two(j), b = raw[i].two(4 + j);
                        float2 va = ffma2(a, k[j], fmul2(b, k[8 + j])), vb = ffma2(b, k[4 + j], fmul2(a, k[12 + j]));
                        if constexpr (kNormed) va = fmul2(va, r2), vb = fmul2(vb, r2);
                        y.set(j, va);
                        y.set(4 + j, vb);
                    }
                }
                if (h < H && th.live) y.store(yt.at(h), th.at);
            }
        }
    }
}

// Gradient of the norm and the rotation.  The grid is what fits on the SMs and
// every warp walks many tokens, all of the queries' first and then all of the
// keys', so that the weight gradients of one side stay in its registers; each
// block leaves its sums (over its warps, in a fixed order) for
// weight_grad_kernel.  A warp loads one pass ahead of the one it computes, over
// the end of a token too; the weights wait in shared memory to make room.  32760
// tokens of 24/24 heads, D = 128, bf16: 233 us, 5.2 TB/s (without the lookahead
// 257; through a ring in shared memory 296).  It issues 2.3 instructions per
// clock of 4 and has 16 warps on an SM: both bound it.
template <typename T, int kStyle, int kBlocks>
__global__ void __launch_bounds__(32 * kGradWarps, kBlocks) norm_grad_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float2 cs_all[kGradWarps][kMaxRopeDim / 2];
    __shared__ float sums[kGradWarps][kMaxRopeDim];
    __shared__ float4 ws[4][32];  // twos 2q, 2q + 1 of group g at [q][g]
    __shared__ uint32_t partners[kStyle == kShifted ? kGradWarps : 1][kStyle == kShifted ? 32 * Partners<T>::kWords : 1];
    const Partners<T> pt{partners[kStyle == kShifted ? warp_id() : 0]};
    griddep_launch_dependents();  // weight_grad_kernel, which waits for this kernel before it reads
    float2* cs = cs_all[warp_id()];
    const RowThread th(p, kStyle);
    const int per_pass = 32 >> p.log2_L;
    const int64_t units = (int64_t)p.B * p.S * p.units_per_token;
    const int64_t step = (int64_t)gridDim.x * kGradWarps, first = (int64_t)blockIdx.x * kGradWarps + warp_id();
    const float inv_d = 1.f / (float)p.D;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        if (p.passes[side] == 0) continue;
        const int H = p.H[side];
        __syncthreads();  // the other side's weights have been read
        if (warp_id() == 0 && th.slot == 0) {
            float2 w[8];
            th.weights(p, side, w);
#pragma unroll
            for (int q = 0; q < 4; ++q) ws[q][lane_id()] = make_float4(w[2 * q].x, w[2 * q].y, w[2 * q + 1].x, w[2 * q + 1].y);
        }
        __syncthreads();
        float2 dw[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = make_float2(0.f, 0.f);

        // a position of the walk: unit un, passes [ps, p1) of it left
        struct Walk {
            int64_t un;
            int b, s, ps, p1;
        };
        auto enter = [&](Walk& w) {  // the first unit from w.un on that has passes of this side
            for (; w.un < units; w.un += step) {
                const Unit u = unit_at(p, w.un);
                w.b = u.b;
                w.s = u.s;
                w.ps = (int)((int64_t)p.passes[side] * u.part / p.units_per_token);
                w.p1 = (int)((int64_t)p.passes[side] * (u.part + 1) / p.units_per_token);
                if (w.ps < w.p1) return;
            }
        };
        auto fetch = [&](const Walk& w, Group<T>& x, Group<T>& g) {
            if (w.un >= units) return;
            const int h = min(w.ps * per_pass + th.slot, H - 1);
            x.load(token_row<T>(p.x[side], w.b, w.s) + h * p.x[side].sh, th.at);
            g.load(token_row<T>(p.g[side], w.b, w.s) + h * p.g[side].sh, th.at);
        };
        Walk ld{first, 0, 0, 0, 0};
        enter(ld);
        Group<T> xn, gn;
        fetch(ld, xn, gn);
        // interleaved: cos, sin of pair j; half: cos of pairs 2j, 2j + 1, then
        // their sines; shifted: cos of elements 2j, 2j + 1, then their signed sines
        float2 c[kStyle == kShifted ? 16 : 8];
        int64_t angles_of = -1;
        while (ld.un < units) {
            const Walk cu = ld;
            const Group<T> x = xn, gr = gn;
            if (++ld.ps == ld.p1) {
                ld.un += step;
                enter(ld);
            }
            fetch(ld, xn, gn);
            if (cu.un != angles_of) {
                angles_of = cu.un;
                token_angles<true, sizeof(T) == 4>(p, Unit{cu.b, cu.s, 0}, cs);
                if constexpr (kStyle == kShifted) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 a0 = th.angle_of(p, cs, th.group * 16 + 2 * j);
                        const float2 a1 = th.angle_of(p, cs, th.group * 16 + 2 * j + 1);
                        c[j] = make_float2(a0.x, a1.x);
                        c[8 + j] = make_float2(-a0.y, -a1.y);  // the transposed rotation
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 a = th.angles(p, cs, j);
                        c[kStyle == kInter ? 2 * j : j] = kStyle == kInter ? make_float2(a.x, a.y) : make_float2(a.x, a.z);
                        c[kStyle == kInter ? 2 * j + 1 : 4 + j] = kStyle == kInter ? make_float2(a.z, a.w) : make_float2(a.y, a.w);
                    }
                }
            }
            const int h = cu.ps * per_pass + th.slot;
            const bool on = h < H;
            float2 g[8];
            if constexpr (kStyle == kShifted) {
                pt.put(gr);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    g[j] = ffma2(gr.two(j), c[j], fmul2(pt.pair(p, th.group * 16 + 2 * j, th.lane0), c[8 + j]));
            } else if constexpr (kStyle == kInter) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 v = gr.two(j);
                    g[j] = make_float2(fmaf(v.x, c[j].x, v.y * c[j].y), fmaf(v.y, c[j].x, -(v.x * c[j].y)));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 g1 = gr.two(j), g2 = gr.two(4 + j);
                    g[j] = ffma2(g1, c[j], fmul2(g2, c[4 + j]));
                    g[4 + j] = fsub2(fmul2(g2, c[j]), fmul2(g1, c[4 + j]));
                }
            }
            float2 q0 = make_float2(0.f, 0.f), q1 = q0, gq0 = q0, gq1 = q0;
            float2 gw[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 x0 = x.two(j), x1 = x.two(j + 1);
                const float4 w = ws[j / 2][th.group];
                gw[j] = fmul2(g[j], make_float2(w.x, w.y));
                gw[j + 1] = fmul2(g[j + 1], make_float2(w.z, w.w));
                q0 = ffma2(x0, x0, q0);
                q1 = ffma2(x1, x1, q1);
                gq0 = ffma2(gw[j], x0, gq0);
                gq1 = ffma2(gw[j + 1], x1, gq1);
            }
            q0 = fadd2(q0, q1);
            gq0 = fadd2(gq0, gq1);
            float sums2[2] = {q0.x + q0.y, gq0.x + gq0.y};  // x^2, g w x
            th.row_sums(p, sums2);
            const float r = on ? row_rsqrt<T>(fmaf(sums2[0], inv_d, p.eps)) : 0.f;
            const float kx = -r * r * r * (sums2[1] * inv_d);
            const float2 r2 = make_float2(r, r), k2 = make_float2(kx, kx);
            Group<T> y;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 xj = x.two(j);
                dw[j] = ffma2(fmul2(g[j], r2), xj, dw[j]);
                y.set(j, ffma2(gw[j], r2, fmul2(xj, k2)));
            }
            if (on && th.live) y.store(token_row<T>(p.y[side], cu.b, cu.s) + h * p.y[side].sh, th.at);
        }
        if (p.dw_part) {
            // over the warp's heads, then over the block's warps, in a fixed order
            __syncthreads();  // the other side's sums have been read
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float va = dw[j].x, vb = dw[j].y;
                for (int o = p.L; o < 32; o <<= 1) {
                    va += __shfl_xor_sync(0xffffffffu, va, o);
                    vb += __shfl_xor_sync(0xffffffffu, vb, o);
                }
                const int e = j < 4 ? th.at.x + 2 * j : th.at.y + 2 * (j - 4);
                if (th.live && th.slot == 0) {
                    sums[warp_id()][e] = va;
                    sums[warp_id()][e + 1] = vb;
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < p.D; i += blockDim.x) {
                float v = 0.f;
#pragma unroll
                for (int wi = 0; wi < kGradWarps; ++wi) v += sums[wi][i];
                p.dw_part[((int64_t)blockIdx.x * 2 + side) * p.D + i] = v;
            }
        }
    }
}

// --------------------------------------------------------- single pairs
// Any even D and rot_dim, any alignment: lane holds pairs lane, lane + 32, ..
// of one head at a time; two-byte (four-byte) accesses.
constexpr int kPairs = kMaxRopeDim / 64;

template <typename T, int kMode>
__global__ void __launch_bounds__(32 * kGradWarps) rope_pairs_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 cs_all[kGradWarps][kMaxRopeDim / 2];
    __shared__ float sums[kMode == kNormGrad ? kGradWarps : 1][kMode == kNormGrad ? kMaxRopeDim : 1];
    if constexpr (kMode == kNormGrad) griddep_launch_dependents();  // weight_grad_kernel
    float2* cs = cs_all[warp_id()];
    const int lane = lane_id(), np = p.D / 2;
    const int64_t units = (int64_t)p.B * p.S * p.units_per_token;
    const float inv_d = 1.f / (float)p.D;
    int2 e[kPairs];  // elements of pair lane + 32 k
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        const int i = min(lane + 32 * k, np - 1);
        e[k] = !p.interleaved && i < p.rot / 2 ? make_int2(i, p.rot / 2 + i) : make_int2(2 * i, 2 * i + 1);
    }
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        if (p.passes[side] == 0) continue;
        float wa[kPairs], wb[kPairs], dwa[kPairs], dwb[kPairs];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            dwa[k] = dwb[k] = 0.f;
            wa[k] = kMode == kRotate ? 1.f : weight_at(p, side, e[k].x);
            wb[k] = kMode == kRotate ? 1.f : weight_at(p, side, e[k].y);
        }
        for (int64_t un = (int64_t)blockIdx.x * kGradWarps + warp_id(); un < units; un += (int64_t)gridDim.x * kGradWarps) {
            const Unit u = unit_at(p, un);
            const int h0 = (int)((int64_t)p.H[side] * u.part / p.units_per_token);
            const int h1 = (int)((int64_t)p.H[side] * (u.part + 1) / p.units_per_token);
            if (h0 >= h1) continue;
            token_angles<false, sizeof(T) == 4>(p, u, cs);
            for (int h = h0; h < h1; ++h) {
                const T* x = token_row<T>(p.x[side], u.b, u.s) + h * p.x[side].sh;
                const T* g = kMode == kNormGrad ? token_row<T>(p.g[side], u.b, u.s) + h * p.g[side].sh : x;
                T* y = token_row<T>(p.y[side], u.b, u.s) + h * p.y[side].sh;
                float a[kPairs], b[kPairs], ga[kPairs], gb[kPairs], sx = 0.f, sgx = 0.f;
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    const int i = lane + 32 * k;
                    const bool on = i < np;
                    a[k] = on ? to_f<T>(x[e[k].x]) : 0.f;
                    b[k] = on ? to_f<T>(x[e[k].y]) : 0.f;
                    sx = fmaf(a[k], a[k], fmaf(b[k], b[k], sx));
                    if constexpr (kMode == kNormGrad) {
                        const float2 v = on ? cs[i] : make_float2(1.f, 0.f);
                        const float g1 = on ? to_f<T>(g[e[k].x]) : 0.f, g2 = on ? to_f<T>(g[e[k].y]) : 0.f;
                        ga[k] = g1 * v.x + g2 * v.y;
                        gb[k] = g2 * v.x - g1 * v.y;
                        sgx = fmaf(ga[k] * wa[k], a[k], fmaf(gb[k] * wb[k], b[k], sgx));
                    }
                }
                float r = 1.f;
                if constexpr (kMode != kRotate) {
                    for (int o = 16; o > 0; o >>= 1) {
                        sx += __shfl_xor_sync(0xffffffffu, sx, o);
                        if (kMode == kNormGrad) sgx += __shfl_xor_sync(0xffffffffu, sgx, o);
                    }
                    r = row_rsqrt<T>(fmaf(sx, inv_d, p.eps));
                }
                const float kx = -r * r * r * (sgx * inv_d);
                // every element has been read: y may be x or g
                __syncwarp();
#pragma unroll
                for (int k = 0; k < kPairs; ++k) {
                    const int i = lane + 32 * k;
                    if (i >= np) continue;
                    float ya, yb;
                    if constexpr (kMode == kNormGrad) {
                        dwa[k] = fmaf(ga[k] * a[k], r, dwa[k]);
                        dwb[k] = fmaf(gb[k] * b[k], r, dwb[k]);
                        ya = fmaf(ga[k] * wa[k], r, a[k] * kx);
                        yb = fmaf(gb[k] * wb[k], r, b[k] * kx);
                    } else {
                        const float2 v = cs[i];
                        const float xa = a[k] * r * wa[k], xb = b[k] * r * wb[k];
                        ya = xa * v.x - xb * v.y;
                        yb = xb * v.x + xa * v.y;
                    }
                    y[e[k].x] = from_f<T>(ya);
                    y[e[k].y] = from_f<T>(yb);
                }
            }
        }
        if (kMode == kNormGrad && p.dw_part) {
            __syncthreads();  // the other side's sums have been read
#pragma unroll
            for (int k = 0; k < kPairs; ++k)
                if (lane + 32 * k < np) {
                    sums[warp_id()][e[k].x] = dwa[k];
                    sums[warp_id()][e[k].y] = dwb[k];
                }
            __syncthreads();
            for (int i = threadIdx.x; i < p.D; i += blockDim.x) {
                float v = 0.f;
#pragma unroll
                for (int wi = 0; wi < kGradWarps; ++wi) v += sums[kMode == kNormGrad ? wi : 0][i];
                p.dw_part[((int64_t)blockIdx.x * 2 + side) * p.D + i] = v;
            }
        }
    }
}

// dw = the sum of the blocks' partial gradients, in a fixed order: 32 columns
// by 32 row groups per block, added as a tree (1.0e-7 of dw's norm off on 5000
// rows of fp32, one after the other 1.5e-7).
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows) weight_grad_kernel(const float* __restrict__ part, int blocks, int D,
                                                                    float* dwq, float* dwk) {
    griddep_wait();  // the gradient kernel is complete (launch_kernel)
    __shared__ float sm[kSumRows][33];
    const int col = blockIdx.x * 32 + threadIdx.x;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (col < 2 * D) {
        for (int i = threadIdx.y; i < blocks; i += 4 * kSumRows) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * kSumRows < blocks) v[k] += part[(int64_t)(i + k * kSumRows) * 2 * D + col];
        }
    }
    sm[threadIdx.y][threadIdx.x] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    // warp y adds column y
    float sum = sm[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int mine = blockIdx.x * 32 + threadIdx.y;
    float* out = mine < D ? dwq : dwk;
    if (threadIdx.x == 0 && mine < 2 * D && out) out[mine < D ? mine : mine - D] = sum;
}

template <typename T, int kMode>
cudaError_t launch_rope_mode(const RopeParams& p, bool vec, unsigned grid, cudaStream_t s) {
    const dim3 blk(32 * kWarps), gblk(32 * kGradWarps);
    const int style = p.interleaved ? kInter : p.rot % 16 == 0 ? kHalf : kShifted;
    if (!vec) return launch_kernel(false, rope_pairs_kernel<T, kMode>, dim3(grid), gblk, 0, s, p);
    if constexpr (kMode == kNormGrad) {
        constexpr int kBlocks = sizeof(T) == 4 ? kGradBlocksWide : kGradBlocks;
        auto kern = style == kInter ? norm_grad_kernel<T, kInter, kBlocks>
                    : style == kHalf ? norm_grad_kernel<T, kHalf, kBlocks>
                                     : norm_grad_kernel<T, kShifted, kGradBlocksWide>;
        return launch_kernel(false, kern, dim3(grid), gblk, 0, s, p);
    } else {
        // Passes in flight against warps on an SM.  The norm's six (the longest
        // batch that does not spill at 16 warps) take 126 us on 32760 tokens
        // of 24/24 heads, D = 128, two at 24 warps 143; rows of fewer passes
        // have nothing to fill six with.
        constexpr bool kNormed = kMode == kNorm;
        constexpr int kLong = sizeof(T) == 4 ? 2 : kNormed ? 6 : 3, kLongBlocks = kNormed ? 8 : 12;
        constexpr int kShort = 2, kShortBlocks = 12;
        //
        // The rotation's passes run over queries' and keys' heads together where
        // that makes fewer of them (20000 tokens of 6/2 heads, D = 128: 18 us, a
        // side at a time 23), and with 16-bit types where they are few, as the
        // factors are then folded once (272440 of 8/2, D = 80: 268 and 288; 30000
        // of 8/8: 41.9 and 43.3; but 20000 of 24/8, eight passes: 53.2 and 51.2,
        // and of 8/8 in fp32 55.5 and 51.7).
        const bool few = kNormed ? std::max(p.passes[0], p.passes[1]) <= 3 : p.joined != 0;
        auto kern = style == kInter ? (few ? rope_kernel<T, kInter, kNormed, !kNormed, kShort, kShortBlocks>
                                           : rope_kernel<T, kInter, kNormed, false, kLong, kLongBlocks>)
                    : style == kHalf ? (few ? rope_kernel<T, kHalf, kNormed, !kNormed, kShort, kShortBlocks>
                                            : rope_kernel<T, kHalf, kNormed, false, kLong, kLongBlocks>)
                                     : rope_kernel<T, kShifted, kNormed, !kNormed, kShort, 8>;
        return launch_kernel(false, kern, dim3(grid), blk, 0, s, p);
    }
}

template <int kMode>
cudaError_t launch_rope(const RopeParams& p, ctx_dtype_t dtype, bool vec, unsigned grid, cudaStream_t s) {
    switch (dtype) {
        case CTX_DTYPE_BF16: return launch_rope_mode<__nv_bfloat16, kMode>(p, vec, grid, s);
        case CTX_DTYPE_FP16: return launch_rope_mode<__half, kMode>(p, vec, grid, s);
        default: return launch_rope_mode<float, kMode>(p, vec, grid, s);
    }
}

bool dtype_ok(int t) { return t == CTX_DTYPE_BF16 || t == CTX_DTYPE_FP16 || t == CTX_DTYPE_FP32; }

// 16-byte accesses at multiples of 8 elements of every row
bool rows_aligned(const Dense& d, int64_t B, int64_t S, int64_t H, int64_t size) {
    const int64_t a = 16 / size;
    return !(reinterpret_cast<uintptr_t>(d.data) & 15) && (B == 1 || d.sb % a == 0) && (S == 1 || d.ss % a == 0) &&
           (H == 1 || d.sh % a == 0);
}

// Arguments common to the four entry points.  x: q and k; g: the incoming
// gradients (backward of the norm only); y: the results.
int rope_call(const char* name, int mode, const ctx_tensor_t* const x[2], const ctx_tensor_t* const g[2],
              const ctx_tensor_t* const y[2], const void* const w[2], int w_dtype, float eps, const ctx_rope_t* rope,
              bool inverse, int dtype, ctx_layout_t layout, float* const dw[2], void* workspace,
              size_t workspace_bytes, ctx_stream_t stream) {
    if (!x[0] || !y[0] || (x[1] == nullptr) != (y[1] == nullptr)) return CTX_ERR_INVALID_ARG;
    if (!x[1] && (w[1] || dw[1])) return CTX_ERR_INVALID_ARG;
    if (layout != CTX_LAYOUT_BSHD && layout != CTX_LAYOUT_SBHD) return CTX_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || (mode != kRotate && !dtype_ok(w_dtype))) return CTX_ERR_INVALID_ARG;
    if (mode != kRotate && !(eps >= 0.f && isfinite(eps))) return CTX_ERR_INVALID_ARG;
    const int64_t B = x[0]->B, S = x[0]->S, D = x[0]->D;
    if (B < 1 || S < 1 || D < 2 || B > INT32_MAX || S > INT32_MAX) return CTX_ERR_INVALID_ARG;
    if (D % 2 || D > kMaxRopeDim) return CTX_ERR_UNSUPPORTED;
    RopeParams p;
    memset(&p, 0, sizeof(p));
    const int64_t size = dtype == CTX_DTYPE_FP32 ? 4 : 2;
    bool aligned = true;
    for (int i = 0; i < 2; ++i) {
        if (!x[i]) continue;
        const int64_t H = x[i]->H;
        if (H < 1 || H > 65535) return CTX_ERR_INVALID_ARG;
        const ctx_tensor_t* t[3] = {x[i], y[i], mode == kNormGrad ? g[i] : nullptr};
        RopeRows* rows[3] = {&p.x[i], &p.y[i], &p.g[i]};
        for (int n = 0; n < (mode == kNormGrad ? 3 : 2); ++n) {
            Dense d;
            const int rc = resolve_strides(t[n], B, S, H, D, layout, &d);
            if (rc) return rc;
            if (reinterpret_cast<uintptr_t>(d.data) % size) return CTX_ERR_UNSUPPORTED;
            aligned = aligned && rows_aligned(d, B, S, H, size);
            rows[n]->p = d.data;
            rows[n]->sb = d.sb; rows[n]->ss = d.ss; rows[n]->sh = d.sh;
        }
        p.H[i] = (int)H;
        p.w[i] = w[i];
        if (w[i] && reinterpret_cast<uintptr_t>(w[i]) % (w_dtype == CTX_DTYPE_FP32 ? 4 : 2)) return CTX_ERR_UNSUPPORTED;
        aligned = aligned && !(reinterpret_cast<uintptr_t>(w[i]) & 15);
        p.dw[i] = dw[i];
        if (dw[i] && (!w[i] || reinterpret_cast<uintptr_t>(dw[i]) % 4)) return CTX_ERR_INVALID_ARG;
    }
    p.B = (int)B; p.S = (int)S; p.D = (int)D;
    p.w_type = w_dtype;
    p.eps = eps;
    p.m = 1.f;
    if (rope) {
        if (!rope->turns || rope->rot_dim < 2 || rope->rot_dim > D || rope->rot_dim % 2) return CTX_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(rope->turns) % 8 || reinterpret_cast<uintptr_t>(rope->positions) % 8)
            return CTX_ERR_UNSUPPORTED;
        if (rope->n_axes < 1 || rope->n_axes > 4 || !isfinite(rope->magnitude)) return CTX_ERR_INVALID_ARG;
        if (rope->n_axes > 1 && !rope->positions) return CTX_ERR_INVALID_ARG;
        int end = 0;
        for (int a = 0; a < rope->n_axes; ++a) {
            const int n = rope->n_axes == 1 ? rope->rot_dim / 2 : rope->sections[a];
            if (n < 1 || n > rope->rot_dim / 2 - end) return CTX_ERR_INVALID_ARG;
            p.sec_end[a] = end += n;
        }
        if (end != rope->rot_dim / 2) return CTX_ERR_INVALID_ARG;
        p.rot = rope->rot_dim;
        p.turns = rope->turns;
        p.pos = rope->positions;
        p.pos_sb = rope->pos_stride_b; p.pos_ss = rope->pos_stride_s; p.pos_sa = rope->pos_stride_axis;
        if (p.pos_sb < 0 || p.pos_ss < 0 || p.pos_sa < 0) return CTX_ERR_INVALID_ARG;
        p.offset = rope->offset;
        p.n_axes = rope->n_axes;
        p.interleaved = rope->interleaved ? 1 : 0;
        p.m = rope->magnitude;
    } else if (mode == kRotate) {
        return CTX_ERR_INVALID_ARG;
    } else {
        p.interleaved = 1;
    }
    p.sin_sign = inverse ? -p.m : p.m;
    const bool vec = aligned && D % 16 == 0;
    int groups = vec ? (int)D / 16 : 32;
    while ((1 << p.log2_L) < groups) ++p.log2_L;
    p.L = 1 << p.log2_L;
    const int per_pass = 32 / p.L;
    for (int i = 0; i < 2; ++i) p.passes[i] = (p.H[i] + per_pass - 1) / per_pass;
    const int together = (p.H[0] + p.H[1] + per_pass - 1) / per_pass;
    const bool shifted = !p.interleaved && p.rot % 16 != 0;
    if (mode == kRotate && vec &&
        (shifted || together < p.passes[0] + p.passes[1] || (size == 2 && together <= kJoinedPasses))) {
        p.joined = 1;
        p.passes[0] = together;
        p.passes[1] = 0;
    }
    const int total = p.passes[0] + p.passes[1];
    const int64_t tokens = B * S;
    const int sms = num_sms();
    // few tokens: their heads are spread over warps so that every SM has work
    int64_t parts = 1;
    while (parts < total && tokens * parts < 16LL * sms) parts *= 2;
    if (parts > total) parts = total;
    p.per_unit = (int)((total + parts - 1) / parts);
    p.units_per_token = (total + p.per_unit - 1) / p.per_unit;
    const int64_t units = tokens * p.units_per_token;
    const bool walk = mode == kNormGrad || !vec;  // kernels whose warps walk many units
    const int warps = walk ? kGradWarps : kWarps;
    int64_t grid = (units + warps - 1) / warps;
    const bool wide = size == 4 || shifted;
    const int64_t per_sm = !vec ? 16 : wide ? kGradBlocksWide : kGradBlocks;
    if (walk) grid = std::min<int64_t>(grid, std::min<int64_t>(per_sm * sms, kMaxGradBlocks));
    if (grid > INT32_MAX) return CTX_ERR_INVALID_ARG;
    const bool want_dw = mode == kNormGrad && (p.dw[0] || p.dw[1]);
    if (want_dw) {
        if (!workspace || workspace_bytes < ctx_qk_norm_rope_workspace_size((int)D) ||
            (reinterpret_cast<uintptr_t>(workspace) & 255))
            return CTX_ERR_WORKSPACE;
        p.dw_part = static_cast<float*>(workspace);
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (log_enabled())
        fprintf(stderr, "%s: B=%d S=%d Hq=%d Hk=%d D=%d rot=%d %s | %s, %lld blocks, %d units per token\n", name, p.B,
                p.S, p.H[0], p.H[1], p.D, p.rot, p.interleaved ? "interleaved" : "half",
                vec ? "16-byte groups" : "single pairs", (long long)grid, p.units_per_token);
    cudaError_t e;
    if (mode == kRotate) e = launch_rope<kRotate>(p, (ctx_dtype_t)dtype, vec, (unsigned)grid, s);
    else if (mode == kNorm) e = launch_rope<kNorm>(p, (ctx_dtype_t)dtype, vec, (unsigned)grid, s);
    else e = launch_rope<kNormGrad>(p, (ctx_dtype_t)dtype, vec, (unsigned)grid, s);
    int rc = launch_status(e);
    if (rc || !want_dw) return rc;
    return launch_status(launch_kernel(!stream_captured(s), weight_grad_kernel, dim3((unsigned)((2 * D + 31) / 32)),
                                       dim3(32, kSumRows), 0, s, (const float*)p.dw_part, (int)grid, (int)D, p.dw[0], p.dw[1]));
}

}  // namespace
}  // namespace ctxattn

using namespace ctxattn;

extern "C" {

size_t ctx_qk_norm_rope_workspace_size(int D) {
    if (D < 2 || D % 2 || D > kMaxRopeDim) return 0;
    return align256((size_t)kMaxGradBlocks * 2 * D * sizeof(float));
}

int ctx_rope_fwd(const ctx_tensor_t* q, const ctx_tensor_t* k, const ctx_rope_t* rope, ctx_dtype_t dtype,
                 ctx_layout_t layout, const ctx_tensor_t* q_out, const ctx_tensor_t* k_out, ctx_stream_t stream) {
    NvtxRange range("ctx_rope_fwd");
    const ctx_tensor_t *x[2] = {q, k}, *y[2] = {q_out, k_out}, *none[2] = {nullptr, nullptr};
    const void* w[2] = {nullptr, nullptr};
    float* dw[2] = {nullptr, nullptr};
    return rope_call("ctx_rope_fwd", kRotate, x, none, y, w, 0, 0.f, rope, false, dtype, layout, dw, nullptr, 0, stream);
}

int ctx_rope_bwd(const ctx_tensor_t* dq_out, const ctx_tensor_t* dk_out, const ctx_rope_t* rope, ctx_dtype_t dtype,
                 ctx_layout_t layout, const ctx_tensor_t* dq, const ctx_tensor_t* dk, ctx_stream_t stream) {
    NvtxRange range("ctx_rope_bwd");
    const ctx_tensor_t *x[2] = {dq_out, dk_out}, *y[2] = {dq, dk}, *none[2] = {nullptr, nullptr};
    const void* w[2] = {nullptr, nullptr};
    float* dw[2] = {nullptr, nullptr};
    return rope_call("ctx_rope_bwd", kRotate, x, none, y, w, 0, 0.f, rope, true, dtype, layout, dw, nullptr, 0, stream);
}

int ctx_qk_norm_rope_fwd(const ctx_tensor_t* q, const ctx_tensor_t* k, const void* wq, const void* wk,
                         ctx_dtype_t w_dtype, float eps, const ctx_rope_t* rope, ctx_dtype_t dtype,
                         ctx_layout_t layout, const ctx_tensor_t* q_out, const ctx_tensor_t* k_out,
                         ctx_stream_t stream) {
    NvtxRange range("ctx_qk_norm_rope_fwd");
    const ctx_tensor_t *x[2] = {q, k}, *y[2] = {q_out, k_out}, *none[2] = {nullptr, nullptr};
    const void* w[2] = {wq, wk};
    float* dw[2] = {nullptr, nullptr};
    return rope_call("ctx_qk_norm_rope_fwd", kNorm, x, none, y, w, w_dtype, eps, rope, false, dtype, layout, dw,
                     nullptr, 0, stream);
}

int ctx_qk_norm_rope_bwd(const ctx_tensor_t* dq_out, const ctx_tensor_t* dk_out, const ctx_tensor_t* q,
                         const ctx_tensor_t* k, const void* wq, const void* wk, ctx_dtype_t w_dtype, float eps,
                         const ctx_rope_t* rope, ctx_dtype_t dtype, ctx_layout_t layout, const ctx_tensor_t* dq,
                         const ctx_tensor_t* dk, float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                         ctx_stream_t stream) {
    NvtxRange range("ctx_qk_norm_rope_bwd");
    if (!dq_out || (k == nullptr) != (dk_out == nullptr)) return CTX_ERR_INVALID_ARG;
    const ctx_tensor_t *x[2] = {q, k}, *g[2] = {dq_out, dk_out}, *y[2] = {dq, dk};
    const void* w[2] = {wq, wk};
    float* dw[2] = {dwq, dwk};
    return rope_call("ctx_qk_norm_rope_bwd", kNormGrad, x, g, y, w, w_dtype, eps, rope, false, dtype, layout, dw,
                     workspace, workspace_bytes, stream);
}

}  // extern "C"

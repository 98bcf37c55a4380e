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
// kernels take the sine and cosine of, in fp32 (2^-24 of half a turn).
// With the norm, y = R(x r w) with r = 1 / sqrt(mean(x^2) + eps); backward
// (g = R^T dy, gw = g w):  dx = r (gw - x r^2 mean(gw x)),  dw = sum g x r.
// Everything between the load and the store is fp32; values are rounded once.
//
// Layout of the work.  A thread holds whole pairs: kVec of them per group, so
// no element crosses threads for the rotation and a row's sums are a shuffle
// over the L lanes that share the head.  A warp takes one token and walks
// passes of 32 / L heads, so the sines and cosines of a token are computed
// once for all of its query and key heads.
//   kVec = 8: two 16-byte accesses (for 16-bit types) per thread and tensor;
//             needs D, R multiples of 16 and 16-byte aligned rows.
//   kVec = 1: any even D and R, any strides.
#include <math.h>
#include <string.h>

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "api_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace ctxattn {
namespace {

constexpr int kMaxRopeDim = 512;
constexpr int kWarps = 8;  // warps of a block
constexpr int kMaxGradBlocks = 1024;  // blocks of the backward that leave partial weight gradients

enum { kRotate = 0, kNorm = 1, kNormGrad = 2 };

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
    float m, sin_sign, eps;
    float* dw_part;             // [blocks][2][D], or null
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

// N consecutive elements as stored (N = 8: 16-byte accesses).
template <typename T, int N>
struct Chunk {
    T e[N];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (N == 8) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) * N / 16; ++i)
                reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
        } else {
            e[0] = *p;
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (N == 8) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) * N / 16; ++i)
                reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(e)[i];
        } else {
            *p = e[0];
        }
    }
};

// Where group g's two chunks of kVec elements start.  Rotated pairs in the
// half layout: g and R/2 + g; otherwise 2 kVec consecutive elements.
template <int kVec>
__device__ __forceinline__ int2 chunk_at(int g, int rot, int interleaved) {
    const bool split = !interleaved && g * kVec < rot / 2;
    return split ? make_int2(g * kVec, rot / 2 + g * kVec) : make_int2(2 * g * kVec, 2 * g * kVec + kVec);
}

// The pairs (a[j], b[j]) of a group, from its two chunks and back.  In the
// interleaved layout (and in the part that is not rotated, where the pairing
// is of no consequence) a pair is two neighbouring elements.
template <typename T, int kVec>
__device__ __forceinline__ void unpack(const Chunk<T, kVec>& c0, const Chunk<T, kVec>& c1, bool inter, float* a,
                                       float* b) {
    if (kVec == 1 || !inter) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            a[j] = to_f<T>(c0.e[j]);
            b[j] = to_f<T>(c1.e[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            a[j] = to_f<T>(2 * j < kVec ? c0.e[(2 * j) % kVec] : c1.e[(2 * j) % kVec]);
            b[j] = to_f<T>(2 * j < kVec ? c0.e[(2 * j + 1) % kVec] : c1.e[(2 * j + 1) % kVec]);
        }
    }
}
template <typename T, int kVec>
__device__ __forceinline__ void pack(Chunk<T, kVec>& c0, Chunk<T, kVec>& c1, bool inter, const float* a,
                                     const float* b) {
    if (kVec == 1 || !inter) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            c0.e[j] = from_f<T>(a[j]);
            c1.e[j] = from_f<T>(b[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            T& ea = 2 * j < kVec ? c0.e[(2 * j) % kVec] : c1.e[(2 * j) % kVec];
            T& eb = 2 * j < kVec ? c0.e[(2 * j + 1) % kVec] : c1.e[(2 * j + 1) % kVec];
            ea = from_f<T>(a[j]);
            eb = from_f<T>(b[j]);
        }
    }
}

__device__ __forceinline__ float weight_at(const RopeParams& p, int side, int i) {
    if (!p.w[side]) return 1.f;
    return p.w_type == CTX_DTYPE_FP32 ? static_cast<const float*>(p.w[side])[i]
         : p.w_type == CTX_DTYPE_FP16 ? __half2float(static_cast<const __half*>(p.w[side])[i])
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(p.w[side])[i]);
}

// kVec pairs per group, kGroups groups per thread (lane + 32 k when kVec = 1).
template <typename T, int kVec, int kGroups, bool kInter, int kMode>
__global__ void __launch_bounds__(32 * kWarps) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int N = kVec * kGroups;
    const int lane = lane_id();
    const int L = p.L, lig = lane & (L - 1), slot = lane >> p.log2_L, heads_per_pass = 32 >> p.log2_L;
    const int ngroups = p.D / (2 * kVec);
    const bool inter = kVec == 1 ? p.interleaved : kInter;
    const int64_t units = (int64_t)p.B * p.S * p.units_per_token;
    const int64_t nwarps = (int64_t)gridDim.x * kWarps;

    int2 at[kGroups];
    bool live[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const int g = lig + k * L;
        live[k] = g < ngroups;
        at[k] = chunk_at<kVec>(live[k] ? g : 0, p.rot, inter);
    }
    // the style of the pairs of a group: tail groups are consecutive elements
    float dwa[kMode == kNormGrad ? 2 : 1][N], dwb[kMode == kNormGrad ? 2 : 1][N];
    if constexpr (kMode == kNormGrad) {
#pragma unroll
        for (int j = 0; j < N; ++j) dwa[0][j] = dwa[1][j] = dwb[0][j] = dwb[1][j] = 0.f;
    }

    for (int64_t u = (int64_t)blockIdx.x * kWarps + warp_id(); u < units; u += nwarps) {
        const int64_t token = u / p.units_per_token;
        const int part = (int)(u - token * p.units_per_token);
        const int b = (int)(token / p.S), s = (int)(token - (int64_t)b * p.S);
        const int first = part * p.per_unit, last = min(first + p.per_unit, p.passes[0] + p.passes[1]);

        float c[N], sn[N];
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const int i = (lig + k * L) * kVec + j;
                c[k * kVec + j] = 1.f;
                sn[k * kVec + j] = 0.f;
                if (i < p.rot / 2) {
                    int axis = 0;
                    for (int a = 0; a + 1 < p.n_axes; ++a) axis += i >= p.sec_end[a];
                    const int64_t at_pos = p.pos ? p.pos[b * p.pos_sb + s * p.pos_ss + axis * p.pos_sa] : p.offset + s;
                    const int32_t turn = (int32_t)(((uint64_t)at_pos * p.turns[i]) >> 32);
                    float si, co;
                    sincospif((float)turn * 4.656612873077393e-10f, &si, &co);  // 2^-31: half turns
                    c[k * kVec + j] = co * p.m;
                    sn[k * kVec + j] = si * p.sin_sign;
                }
            }

        auto side_passes = [&](auto side_c) {
            constexpr int side = decltype(side_c)::value;
            const int p0 = max(first - (side ? p.passes[0] : 0), 0);
            const int p1 = min(last - (side ? p.passes[0] : 0), p.passes[side]);
            float wa[N], wb[N];
            if (kMode != kRotate && p0 < p1) {
#pragma unroll
                for (int k = 0; k < kGroups; ++k)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        int ia = at[k].x + j, ib = at[k].y + j;
                        if (kVec > 1 && inter) ia = at[k].x + 2 * j, ib = ia + 1;
                        wa[k * kVec + j] = live[k] ? weight_at(p, side, ia) : 0.f;
                        wb[k * kVec + j] = live[k] ? weight_at(p, side, ib) : 0.f;
                    }
            }
            for (int ps = p0; ps < p1; ++ps) {
                const int h = ps * heads_per_pass + slot;
                const bool on = h < p.H[side];
                auto row = [&](const RopeRows& r) { return (T*)r.p + b * r.sb + s * r.ss + (int64_t)(on ? h : 0) * r.sh; };
                Chunk<T, kVec> x0[kGroups], x1[kGroups], g0[kGroups], g1[kGroups];
                float a[N], bb[N];
                const T* xr = row(p.x[side]);
#pragma unroll
                for (int k = 0; k < kGroups; ++k) {
#pragma unroll
                    for (int j = 0; j < kVec; ++j) a[k * kVec + j] = bb[k * kVec + j] = 0.f;
                    if (on && live[k]) {
                        x0[k].load(xr + at[k].x);
                        x1[k].load(xr + at[k].y);
                    }
                }
                if constexpr (kMode == kNormGrad) {
                    const T* gr = row(p.g[side]);
#pragma unroll
                    for (int k = 0; k < kGroups; ++k)
                        if (on && live[k]) {
                            g0[k].load(gr + at[k].x);
                            g1[k].load(gr + at[k].y);
                        }
                }
#pragma unroll
                for (int k = 0; k < kGroups; ++k)
                    if (on && live[k]) unpack<T, kVec>(x0[k], x1[k], inter, a + k * kVec, bb + k * kVec);
                float ya[N], yb[N];
                if constexpr (kMode == kNormGrad) {
                    float ga[N], gb[N], sx = 0.f, sgx = 0.f;
#pragma unroll
                    for (int k = 0; k < kGroups; ++k) {
#pragma unroll
                        for (int j = 0; j < kVec; ++j) ga[k * kVec + j] = gb[k * kVec + j] = 0.f;
                        if (on && live[k]) unpack<T, kVec>(g0[k], g1[k], inter, ga + k * kVec, gb + k * kVec);
                    }
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float t = ga[j];
                        ga[j] = t * c[j] + gb[j] * sn[j];
                        gb[j] = gb[j] * c[j] - t * sn[j];
                        sx = fmaf(a[j], a[j], fmaf(bb[j], bb[j], sx));
                        sgx = fmaf(ga[j] * wa[j], a[j], fmaf(gb[j] * wb[j], bb[j], sgx));
                    }
                    for (int o = L >> 1; o > 0; o >>= 1) {
                        sx += __shfl_xor_sync(0xffffffffu, sx, o);
                        sgx += __shfl_xor_sync(0xffffffffu, sgx, o);
                    }
                    const float r = on ? __frsqrt_rn(sx / (float)p.D + p.eps) : 0.f;
                    const float mean = r * r * (sgx / (float)p.D);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        dwa[side][j] = fmaf(ga[j], a[j] * r, dwa[side][j]);
                        dwb[side][j] = fmaf(gb[j], bb[j] * r, dwb[side][j]);
                        ya[j] = r * (ga[j] * wa[j] - a[j] * mean);
                        yb[j] = r * (gb[j] * wb[j] - bb[j] * mean);
                    }
                } else {
                    if constexpr (kMode == kNorm) {
                        float sx = 0.f;
#pragma unroll
                        for (int j = 0; j < N; ++j) sx = fmaf(a[j], a[j], fmaf(bb[j], bb[j], sx));
                        for (int o = L >> 1; o > 0; o >>= 1) sx += __shfl_xor_sync(0xffffffffu, sx, o);
                        const float r = __frsqrt_rn(sx / (float)p.D + p.eps);
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            a[j] *= r * wa[j];
                            bb[j] *= r * wb[j];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        ya[j] = a[j] * c[j] - bb[j] * sn[j];
                        yb[j] = bb[j] * c[j] + a[j] * sn[j];
                    }
                }
                T* yr = row(p.y[side]);
#pragma unroll
                for (int k = 0; k < kGroups; ++k)
                    if (on && live[k]) {
                        Chunk<T, kVec> o0, o1;
                        pack<T, kVec>(o0, o1, inter, ya + k * kVec, yb + k * kVec);
                        o0.store(yr + at[k].x);
                        o1.store(yr + at[k].y);
                    }
            }
        };
        side_passes(std::integral_constant<int, 0>{});
        side_passes(std::integral_constant<int, 1>{});
    }

    if constexpr (kMode == kNormGrad) {
        if (p.dw_part) {
            // sums over the warp's heads, then over the block's warps, in a fixed order
            __shared__ float sm[kWarps][2 * kMaxRopeDim];
            const int w = warp_id();
#pragma unroll
            for (int side = 0; side < 2; ++side)
#pragma unroll
                for (int k = 0; k < kGroups; ++k)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        float va = dwa[side][k * kVec + j], vb = dwb[side][k * kVec + j];
                        for (int o = L; o < 32; o <<= 1) {
                            va += __shfl_xor_sync(0xffffffffu, va, o);
                            vb += __shfl_xor_sync(0xffffffffu, vb, o);
                        }
                        int ia = at[k].x + j, ib = at[k].y + j;
                        if (kVec > 1 && inter) ia = at[k].x + 2 * j, ib = ia + 1;
                        if (live[k] && slot == 0) {
                            sm[w][side * p.D + ia] = va;
                            sm[w][side * p.D + ib] = vb;
                        }
                    }
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * p.D; i += blockDim.x) {
                float v = 0.f;
#pragma unroll
                for (int ww = 0; ww < kWarps; ++ww) v += sm[ww][i];
                p.dw_part[(int64_t)blockIdx.x * 2 * p.D + i] = v;
            }
        }
    }
}

// dw = the sum of the blocks' partial gradients, in a fixed order: 32 columns
// by 16 row groups per block.
__global__ void weight_grad_kernel(const float* __restrict__ part, int blocks, int D, float* dwq, float* dwk) {
    __shared__ float sm[16][33];
    const int col = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (col < 2 * D)
        for (int i = threadIdx.y; i < blocks; i += 16) v += part[(int64_t)i * 2 * D + col];
    sm[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && col < 2 * D) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += sm[i][threadIdx.x];
        float* out = col < D ? dwq : dwk;
        if (out) out[col < D ? col : col - D] = v;
    }
}

template <typename T, int kMode>
cudaError_t launch_rope_mode(const RopeParams& p, bool vec, unsigned grid, cudaStream_t s) {
    const dim3 blk(32 * kWarps);
    if (vec)
        return p.interleaved ? launch_kernel(false, rope_kernel<T, 8, 1, true, kMode>, dim3(grid), blk, 0, s, p)
                             : launch_kernel(false, rope_kernel<T, 8, 1, false, kMode>, dim3(grid), blk, 0, s, p);
    return launch_kernel(false, rope_kernel<T, 1, kMaxRopeDim / 64, false, kMode>, dim3(grid), blk, 0, s, p);
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
    const bool vec = aligned && D % 16 == 0 && p.rot % 16 == 0;
    int groups = vec ? (int)D / 16 : 32;
    while ((1 << p.log2_L) < groups) ++p.log2_L;
    p.L = 1 << p.log2_L;
    const int per_pass = 32 / p.L;
    for (int i = 0; i < 2; ++i) p.passes[i] = (p.H[i] + per_pass - 1) / per_pass;
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
    int64_t grid = (units + kWarps - 1) / kWarps;
    if (mode == kNormGrad) {
        int64_t cap = 2LL * sms;
        if (cap > kMaxGradBlocks) cap = kMaxGradBlocks;
        if (grid > cap) grid = cap;
    } else if (grid > (1LL << 30)) {
        grid = 1LL << 30;
    }
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
    weight_grad_kernel<<<(unsigned)((2 * D + 31) / 32), dim3(32, 16), 0, s>>>(p.dw_part, (int)grid, (int)D, p.dw[0],
                                                                             p.dw[1]);
    return launch_status();
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

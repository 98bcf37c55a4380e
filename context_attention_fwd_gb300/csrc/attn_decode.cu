// attn_decode.cu -- attention of the newest T tokens of every sequence over
// its key/value cache, causal, under an optional sliding window with sinks.
//
// Mathematics.  Query t of T stands at position p = length - T + t and sees
// key j iff j <= p and (j < sinks or j >= p - left).  Softmax over the visible
// keys with a running maximum m and sum l per row (base 2, fp32), the
// probabilities rounded to bf16 for the product with V (2^-8 of each, as in
// the other attention kernels), O in fp32.
//
// What bounds it: every visible key and value is read once, 4 D bytes a key
// and kv head, so HBM for any real batch.  Hence:
//   * one CTA serves all query rows that share a kv head (the G heads of its
//     group and the T tokens: rows r = t G + g, 16 at a time), so the cache is
//     read once per group, not once per query head;
//   * the keys that some row sees are numbered without gaps, v = 0 .. n - 1
//     (the sinks, then the window), and cut over `splits` CTAs and then over
//     the CTA's four warps in tiles of 8 KB.  Every warp streams its own
//     tiles through its own ring of cp.async slots and keeps its own (m, l,
//     O), so no barrier stands in the loop; keys past n are zero-filled, never
//     read;
//   * products on the warp-level tensor instruction (m16n8k16): a decode step
//     has 16 rows or fewer per kv head, far from what would fill a 128-row
//     tile, and is nowhere near bound by it.
// The warps' states are merged in shared memory; with splits > 1 the CTAs'
// merged states go to the workspace and decode_merge_kernel joins them.  One
// sequence of 65536 tokens, 32/8 heads, D = 128: 44 us, 6.1 TB/s; 64 sequences,
// window 1024, 24/4 heads, D = 256: 42 us, 6.5 TB/s.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "api_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace ctxattn {
namespace {

constexpr int kDecWarps = 4;
constexpr int kRows = 16;  // query rows of a CTA
constexpr int kMaxSplits = 128;

struct DecParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* out;
    float* lse;          // [B,Hq,T]
    const int* lengths;  // [B], or null: cap
    int64_t q_sb, q_ss, q_sh, k_sb, k_ss, k_sh, v_sb, v_ss, v_sh, o_sb, o_ss, o_sh;
    int B, T, Hq, Hkv, G, cap, left, sinks, splits, row_blocks;
    float scale, scale_log2;
    float* part_o;   // [splits][B][Hkv][row_blocks][16][D], not normalised
    float2* part_ml; // [splits][B][Hkv][row_blocks][16]: m (log2 units), l
};

template <int D>
struct DecLayout {
    static constexpr int KEYS = 4096 / D;                // keys of a warp's tile: 8 KB of K, 8 KB of V
    static constexpr int SLOTS = 3;                      // of 8 KB, K and V tiles in turn; two CTAs per SM
    static constexpr uint32_t ROW = D * 2;               // bytes
    static constexpr uint32_t SLOT = KEYS * ROW;
    static constexpr uint32_t OFF_Q = 0;                 // 16 x D bf16
    static constexpr uint32_t OFF_RING = kRows * ROW;
    static constexpr uint32_t SMEM = OFF_RING + kDecWarps * SLOTS * SLOT;
    static_assert(kDecWarps * kRows * (D + 4) * 4 + kDecWarps * kRows * 8 <= SMEM, "merge buffers reuse the ring");
};

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// c[16x8] += a[16x16] b[16x8], bf16 in, fp32 out
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte chunk c of row r: chunks are XORed with r mod 8, so
// that eight rows of one chunk column lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t dec_off(uint32_t r, uint32_t c) {
    return r * (D * 2) + ((c ^ (r & 7u)) << 4);
}

// The keys that some row of a sequence sees, numbered without gaps.
struct DecSpan {
    int len;    // cached tokens
    int n;      // visible keys
    int ns;     // the first ns are sinks before the window
    int shift;  // key = v < ns ? v : v + shift
};
__device__ __forceinline__ DecSpan dec_span(const DecParams& p, int b) {
    DecSpan s;
    s.len = p.lengths ? min(max(p.lengths[b], 0), p.cap) : p.cap;
    const int64_t first = (int64_t)s.len - p.T - p.left;  // of the first token's window
    const int lo = p.left < 0 || first < 0 ? 0 : (int)min(first, (int64_t)s.len);
    s.ns = min(p.sinks, lo);
    s.shift = lo - s.ns;
    s.n = s.len - s.shift;
    return s;
}

template <int D>
__global__ void __launch_bounds__(32 * kDecWarps, 2) attn_decode_kernel(const __grid_constant__ DecParams p) {
    using L = DecLayout<D>;
    constexpr int KEYS = L::KEYS, NT = KEYS / 8, CH = D / 8;
    griddep_launch_dependents();  // decode_merge_kernel, which waits for this kernel before it reads
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = warp_id(), lane = lane_id();
    const int split = blockIdx.x, b = blockIdx.z;
    const int hk = blockIdx.y / p.row_blocks, rb = blockIdx.y % p.row_blocks;
    const int rows = min(kRows, p.T * p.G - rb * kRows);
    const DecSpan sp = dec_span(p, b);
    const int ntiles = (sp.n + KEYS - 1) / KEYS;
    const int t0 = (int)((int64_t)ntiles * split / p.splits), t1 = (int)((int64_t)ntiles * (split + 1) / p.splits);

    // Q rows (zero past the last)
    for (int i = threadIdx.x; i < kRows * CH; i += blockDim.x) {
        const int r = i / CH, c = i % CH, rr = rb * kRows + r;
        const bool on = r < rows;
        const int t = on ? rr / p.G : 0, h = hk * p.G + (on ? rr % p.G : 0);
        cp_async16(sbase + L::OFF_Q + dec_off<D>(r, c), p.q + b * p.q_sb + t * p.q_ss + h * p.q_sh + c * 8, on);
    }
    cp_async_commit();

    const uint32_t ring = sbase + L::OFF_RING + warp * L::SLOTS * L::SLOT;
    const __nv_bfloat16* kb = p.k + b * p.k_sb + hk * p.k_sh;
    const __nv_bfloat16* vb = p.v + b * p.v_sb + hk * p.v_sh;
    // This warp's tiles are t0 + warp, t0 + warp + 4, ..; load n is the K (n
    // even) or V tile of the n / 2-th of them, and goes to slot n mod 3.  A
    // thread copies chunk lc of rows lr, lr + kStep, ..; kStep divides 8, so
    // the row's part of the swizzle is an exclusive or with a constant.
    constexpr int kStep = 32 / CH;
    const int lr = lane / CH, lc = lane % CH;
    const uint32_t dst0 = lr * L::ROW + ((lc ^ lr) << 4);
    auto load = [&](int n, int slot) {
        const int tile = t0 + warp + (n >> 1) * kDecWarps;
        if (tile < t1) {
            const __nv_bfloat16* base = ((n & 1) ? vb : kb) + lc * 8;
            const int64_t ss = (n & 1) ? p.v_ss : p.k_ss;
            const uint32_t dst = ring + slot * L::SLOT;
            const int v0 = tile * KEYS;
            if (v0 >= sp.ns && v0 + KEYS <= sp.n) {  // whole, past the sinks: consecutive rows
                const __nv_bfloat16* src = base + (v0 + sp.shift + lr) * ss;
#pragma unroll
                for (int i = 0; i < KEYS / kStep; ++i) {
                    cp_async16(dst + (dst0 ^ (((i * kStep) & 7) << 4)) + i * kStep * L::ROW, src, true);
                    src += kStep * ss;
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < KEYS / kStep; ++i) {
                    const int v = v0 + i * kStep + lr;
                    const bool on = v < sp.n;
                    const int64_t key = on ? (v < sp.ns ? v : v + sp.shift) : 0;
                    cp_async16(dst + (dst0 ^ (((i * kStep) & 7) << 4)) + i * kStep * L::ROW, base + key * ss, on);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < L::SLOTS; ++i) load(i, i);

    cp_async_wait<L::SLOTS>();
    __syncthreads();
    uint32_t qf[D == 256 ? 1 : D / 16][4];  // D = 256 reads them again for every tile: the registers hold O
    const uint32_t q_addr = sbase + L::OFF_Q;
    if constexpr (D != 256) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) ldsm4(qf[kk], q_addr + dec_off<D>(lane & 15, 2 * kk + (lane >> 4)));
    }

    const int g = lane >> 2, tq = lane & 3;
    int pos[2];  // positions of this thread's two rows
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = rb * kRows + g + 8 * e;
        pos[e] = g + 8 * e < rows ? sp.len - p.T + r / p.G : -1;
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    int slot = 0, n_load = L::SLOTS;
    auto next_slot = [&] { slot = slot + 1 == L::SLOTS ? 0 : slot + 1; };
    for (int tile = t0 + warp; tile < t1; tile += kDecWarps) {
        cp_async_wait<L::SLOTS - 1>();
        __syncwarp();
        const uint32_t ks = ring + slot * L::SLOT;
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t qa[4];
            if constexpr (D == 256) ldsm4(qa, q_addr + dec_off<D>(lane & 15, 2 * kk + (lane >> 4)));
            const uint32_t* a = D == 256 ? qa : qf[D == 256 ? 0 : kk];
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t kf[4];
                ldsm4(kf, ks + dec_off<D>(n * 8 + ((lane >> 4) << 3) + (lane & 7), 2 * kk + ((lane >> 3) & 1)));
                mma16816(s[n], a, kf[0], kf[1]);
                mma16816(s[n + 1], a, kf[2], kf[3]);
            }
        }
        __syncwarp();  // every thread has read the K tile
        load(n_load++, slot);
        next_slot();
        // with one token every loaded key is visible to every row
        const int v0 = tile * KEYS;
        if (p.T > 1 || v0 + KEYS > sp.n) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int v = v0 + n * 8 + 2 * tq + (e & 1);
                    const int j = v < sp.ns ? v : v + sp.shift;
                    const int pr = pos[e >> 1];
                    if (!(v < sp.n && j <= pr && (p.left < 0 || j < p.sinks || j >= pr - p.left))) s[n][e] = -INFINITY;
                }
        }
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[0][2 * e], s[0][2 * e + 1]);
#pragma unroll
            for (int n = 1; n < NT; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * e], s[n][2 * e + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[e], mx * p.scale_log2);
            const float ref = mn == -INFINITY ? 0.f : mn;  // no key yet
            alpha[e] = ex2(m[e] - ref);
            m[e] = mn;
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                s[n][2 * e] = ex2(fmaf(s[n][2 * e], p.scale_log2, -ref));
                s[n][2 * e + 1] = ex2(fmaf(s[n][2 * e + 1], p.scale_log2, -ref));
                sum += s[n][2 * e] + s[n][2 * e + 1];
            }
            l[e] = l[e] * alpha[e] + sum;  // this thread's columns; summed over the quad at the end
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= alpha[0];
            o[i][1] *= alpha[0];
            o[i][2] *= alpha[1];
            o[i][3] *= alpha[1];
        }
        cp_async_wait<L::SLOTS - 1>();
        __syncwarp();
        const uint32_t vs = ring + slot * L::SLOT;
#pragma unroll
        for (int kk = 0; kk < KEYS / 16; ++kk) {
            const uint32_t a[4] = {pack_bf16x2(s[2 * kk][0], s[2 * kk][1]), pack_bf16x2(s[2 * kk][2], s[2 * kk][3]),
                                   pack_bf16x2(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                                   pack_bf16x2(s[2 * kk + 1][2], s[2 * kk + 1][3])};
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t vf[4];
                ldsm4_t(vf, vs + dec_off<D>(kk * 16 + (lane & 15), 2 * i + (lane >> 4)));
                mma16816(o[2 * i], a, vf[0], vf[1]);
                mma16816(o[2 * i + 1], a, vf[2], vf[3]);
            }
        }
        __syncwarp();  // every thread has read the V tile
        load(n_load++, slot);
        next_slot();
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }

    // merge of the four warps' states, through the ring's memory
    cp_async_wait<0>();
    __syncthreads();
    constexpr int PITCH = D + 4;  // floats
    float* so = reinterpret_cast<float*>(smem);
    float2* sml = reinterpret_cast<float2*>(smem + kDecWarps * kRows * PITCH * 4);
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(so + (warp * kRows + g + 8 * e) * PITCH + i * 8 + 2 * tq) =
                make_float2(o[i][2 * e], o[i][2 * e + 1]);
    if (tq == 0) {
        sml[warp * kRows + g] = make_float2(m[0], l[0]);
        sml[warp * kRows + g + 8] = make_float2(m[1], l[1]);
    }
    __syncthreads();
    constexpr int C4 = D / 4;
    for (int i = threadIdx.x; i < rows * C4; i += blockDim.x) {
        const int r = i / C4, c = i % C4, rr = rb * kRows + r;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, sml[w * kRows + r].x);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            const float2 ml = sml[w * kRows + r];
            const float f = ex2(ml.x - ref);
            const float4 x = *reinterpret_cast<const float4*>(so + (w * kRows + r) * PITCH + c * 4);
            ll = fmaf(ml.y, f, ll);
            acc.x = fmaf(x.x, f, acc.x); acc.y = fmaf(x.y, f, acc.y);
            acc.z = fmaf(x.z, f, acc.z); acc.w = fmaf(x.w, f, acc.w);
        }
        if (p.splits > 1) {
            const int64_t row = ((((int64_t)split * p.B + b) * p.Hkv + hk) * p.row_blocks + rb) * kRows + r;
            *reinterpret_cast<float4*>(p.part_o + row * D + c * 4) = acc;
            if (c == 0) p.part_ml[row] = make_float2(mm, ll);
        } else {
            const int t = rr / p.G, h = hk * p.G + rr % p.G;
            const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);  // a row without keys gives 0, NaN stays
            *reinterpret_cast<uint2*>(p.out + b * p.o_sb + t * p.o_ss + h * p.o_sh + c * 4) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            if (c == 0)
                p.lse[((int64_t)b * p.Hq + h) * p.T + t] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
        }
    }
}

// out, lse of one query row per block from the splits' states.  Every warp
// holds all the splits' weights (split 32 i + lane in register i), adds the
// splits warp, warp + 4, .. and the warps' sums are added in order.
template <int D>
__global__ void __launch_bounds__(32 * kDecWarps) decode_merge_kernel(const __grid_constant__ DecParams p) {
    griddep_wait();  // the previous kernel in the stream is complete (launch_kernel)
    constexpr int N = D / 32;
    __shared__ float sm[kDecWarps][D];
    const int lane = lane_id(), warp = warp_id(), per = p.T * p.G;
    const int rr = (int)(blockIdx.x % per);
    const int64_t bh = blockIdx.x / per;
    const int hk = (int)(bh % p.Hkv), b = (int)(bh / p.Hkv);
    const int64_t stride = (int64_t)p.B * p.Hkv * p.row_blocks * kRows;
    const int64_t row = bh * p.row_blocks * kRows + rr;
    float f[kMaxSplits / 32], ll = 0.f, mm = -INFINITY;
    float2 ml[kMaxSplits / 32];
#pragma unroll
    for (int i = 0; i < kMaxSplits / 32; ++i) {
        const int s = 32 * i + lane;
        ml[i] = s < p.splits ? p.part_ml[s * stride + row] : make_float2(-INFINITY, 0.f);
        mm = fmaxf(mm, ml[i].x);
    }
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int i = 0; i < kMaxSplits / 32; ++i) {
        f[i] = ex2(ml[i].x - ref);
        ll = fmaf(ml[i].y, f[i], ll);
    }
    for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, o);
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxSplits / 32; ++i) {
        if (32 * i >= p.splits) break;
#pragma unroll
        for (int e = 0; e < 32; e += kDecWarps) {
            const int s = 32 * i + e + warp;
            const float w = __shfl_sync(0xffffffffu, f[i], e + warp);
            if (s < p.splits) {
                const float* src = p.part_o + (s * stride + row) * D + lane * N;
                float x[N];
                if constexpr (N == 2) {
                    *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
                } else {
#pragma unroll
                    for (int k = 0; k < N; k += 4) *reinterpret_cast<float4*>(x + k) = *reinterpret_cast<const float4*>(src + k);
                }
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] = fmaf(x[k], w, acc[k]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) sm[warp][lane * N + k] = acc[k];
    __syncthreads();
    const int t = rr / p.G, h = hk * p.G + rr % p.G;
    const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
    __nv_bfloat16* dst = p.out + b * p.o_sb + t * p.o_ss + h * p.o_sh;
    for (int i = threadIdx.x; i < D / 2; i += blockDim.x) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            x += sm[w][2 * i];
            y += sm[w][2 * i + 1];
        }
        *reinterpret_cast<uint32_t*>(dst + 2 * i) = pack_bf16x2(x * inv, y * inv);
    }
    if (threadIdx.x == 0)
        p.lse[((int64_t)b * p.Hq + h) * p.T + t] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
}

// Splits of a call: one CTA per SM, no more than there are tiles for all four
// warps of each at the longest length the cache allows.  (Two CTAs fit on an
// SM, but twice the splits cost more in the join than they bring: 47.0
// against 44.0 us for a 65536-token history of 32/8 heads, D = 128.)
int plan_splits(int64_t ctas, int D, int cap, int T, int left, int sinks) {
    int64_t span = cap;
    if (left >= 0) span = std::min(span, (int64_t)left + T + sinks);
    const int keys = 4096 / D * kDecWarps;
    const int64_t most = std::min<int64_t>(kMaxSplits, (span + keys - 1) / keys);
    const int64_t want = num_sms() / ctas;
    return (int)std::max<int64_t>(1, std::min(want, most));
}

bool decode_sizes_ok(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t cap) {
    return B >= 1 && T >= 1 && Hq >= 1 && Hkv >= 1 && cap >= 1 && Hq % Hkv == 0 && B <= 65535 && T <= 65535 &&
           Hq <= 65535 && cap <= INT32_MAX && B * Hq * T <= INT32_MAX && Hkv * ((T * (Hq / Hkv) + kRows - 1) / kRows) <= 65535;
}

size_t decode_ws_bytes(int B, int T, int Hq, int Hkv, int D, int splits) {
    if (splits <= 1) return 0;
    const size_t rows = (size_t)splits * B * Hkv * ((T * (Hq / Hkv) + kRows - 1) / kRows) * kRows;
    return align256(rows * D * 4) + align256(rows * 8);
}

template <int D>
int launch_decode(const DecParams& p, bool pdl, cudaStream_t s) {
    using L = DecLayout<D>;
    static OncePerDevice attr;
    if (!attr.run([] {
            return cudaFuncSetAttribute(attn_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM) ==
                   cudaSuccess;
        }))
        return CTX_ERR_CUDA;
    int rc = launch_status(launch_kernel(false, attn_decode_kernel<D>, dim3(p.splits, p.Hkv * p.row_blocks, p.B),
                                         dim3(32 * kDecWarps), L::SMEM, s, p));
    if (rc || p.splits == 1) return rc;
    return launch_status(launch_kernel(pdl, decode_merge_kernel<D>, dim3((unsigned)((int64_t)p.B * p.Hq * p.T)),
                                       dim3(32 * kDecWarps), 0, s, p));
}

}  // namespace
}  // namespace ctxattn

using namespace ctxattn;

extern "C" {

size_t ctx_attn_decode_workspace_size(int B, int T, int Hq, int Hkv, int D, int capacity, int window_left, int sinks) {
    if (!decode_sizes_ok(B, T, Hq, Hkv, capacity) || (D != 64 && D != 128 && D != 256) || window_left < -1 || sinks < 0)
        return 0;
    const int64_t blocks = (int64_t)B * Hkv * (((int64_t)T * (Hq / Hkv) + kRows - 1) / kRows);
    return decode_ws_bytes(B, T, Hq, Hkv, D, plan_splits(blocks, D, capacity, T, std::min(window_left, capacity),
                                                                  std::min(sinks, capacity)));
}

int ctx_attn_decode(const ctx_tensor_t* q, const ctx_tensor_t* k, const ctx_tensor_t* v, const int* lengths,
                    ctx_layout_t layout, int window_left, int sinks, float scale, const ctx_tensor_t* out, float* lse,
                    void* workspace, size_t workspace_bytes, ctx_stream_t stream) {
    NvtxRange range("ctx_attn_decode");
    if (!q || !k || !v || !out || !lse) return CTX_ERR_INVALID_ARG;
    if (layout != CTX_LAYOUT_BSHD && layout != CTX_LAYOUT_SBHD) return CTX_ERR_INVALID_ARG;
    if (window_left < -1 || sinks < 0) return CTX_ERR_INVALID_ARG;
    const int64_t B = q->B, T = q->S, Hq = q->H, D = q->D, Hkv = k->H, cap = k->S;
    if (!decode_sizes_ok(B, T, Hq, Hkv, cap)) return CTX_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return CTX_ERR_UNSUPPORTED;
    Dense tq, tk, tv, to;
    int rc;
    if ((rc = resolve(q, B, T, Hq, D, layout, &tq))) return rc;
    if ((rc = resolve(k, B, cap, Hkv, D, layout, &tk))) return rc;
    if ((rc = resolve(v, B, cap, Hkv, D, layout, &tv))) return rc;
    if ((rc = resolve(out, B, T, Hq, D, layout, &to))) return rc;
    if ((reinterpret_cast<uintptr_t>(lse) & 3) || (reinterpret_cast<uintptr_t>(lengths) & 3)) return CTX_ERR_INVALID_ARG;
    DecParams p;
    memset(&p, 0, sizeof(p));
    p.q = static_cast<const __nv_bfloat16*>(tq.data);
    p.k = static_cast<const __nv_bfloat16*>(tk.data);
    p.v = static_cast<const __nv_bfloat16*>(tv.data);
    p.out = static_cast<__nv_bfloat16*>(to.data);
    p.lse = lse;
    p.lengths = lengths;
    p.q_sb = tq.sb; p.q_ss = tq.ss; p.q_sh = tq.sh;
    p.k_sb = tk.sb; p.k_ss = tk.ss; p.k_sh = tk.sh;
    p.v_sb = tv.sb; p.v_ss = tv.ss; p.v_sh = tv.sh;
    p.o_sb = to.sb; p.o_ss = to.ss; p.o_sh = to.sh;
    p.B = (int)B; p.T = (int)T; p.Hq = (int)Hq; p.Hkv = (int)Hkv; p.G = (int)(Hq / Hkv);
    p.cap = (int)cap; p.left = std::min(window_left, p.cap); p.sinks = std::min(sinks, p.cap);
    p.row_blocks = (p.T * p.G + kRows - 1) / kRows;
    p.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)D);
    p.scale_log2 = p.scale * 1.4426950408889634f;
    p.splits = plan_splits(B * Hkv * p.row_blocks, (int)D, p.cap, p.T, p.left, p.sinks);
    const size_t need = decode_ws_bytes(p.B, p.T, p.Hq, p.Hkv, (int)D, p.splits);
    if (need) {
        if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255))
            return CTX_ERR_WORKSPACE;
        const size_t rows = (size_t)p.splits * B * Hkv * p.row_blocks * kRows;
        p.part_o = static_cast<float*>(workspace);
        p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + align256(rows * D * 4));
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (log_enabled())
        fprintf(stderr, "ctx_attn_decode: B=%d T=%d Hq=%d Hkv=%d D=%d capacity=%d window=%d sinks=%d | %d splits, %lld CTAs\n",
                p.B, p.T, p.Hq, p.Hkv, (int)D, p.cap, p.left, p.sinks, p.splits,
                (long long)p.splits * p.Hkv * p.row_blocks * p.B);
    // the merge kernel's launch overlaps the first kernel, but not in a stream
    // that is being captured (replaying a graph removes the gap already)
    const bool pdl = !stream_captured(s);
    if (D == 64) return launch_decode<64>(p, pdl, s);
    if (D == 128) return launch_decode<128>(p, pdl, s);
    return launch_decode<256>(p, pdl, s);
}

}  // extern "C"

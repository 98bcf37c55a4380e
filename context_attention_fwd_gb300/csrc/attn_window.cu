// attn_window.cu -- forward of attention under a sliding window with sink
// tokens, head dimensions 64 and 128, for sm_103a.
//
// Mathematics as in attn_fwd.cu: online softmax over the 128-row KV tiles a
// query tile meets (base 2, fp32 statistics, lazy rescale of O), P rounded to
// bf16 for the product with V.  What differs is how little a CTA has to do: a
// query tile meets window / 128 + 1 KV tiles (and those that hold sinks), some
// ten to twenty microseconds of work.  With the two-tile CTAs of attn_fwd.cu,
// one per SM, starting a CTA and writing its output took 8.7 us of 33 at a
// window of 1024, and of the pair's window / 128 + 2 KV tiles each query tile
// had no part in one.  So here a CTA owns one 128-row query tile and half an
// SM: 256 TMEM columns, half the shared memory; while one of the two resident
// CTAs starts or ends, the other computes.  The price is that K and V are
// loaded once per query tile instead of once per two.
//
// Warp roles (192 threads):
//   warp 0     TMA producer of Q (once) and the K tiles
//   warp 1     TMA producer of the V tiles; TMEM owner
//   warps 2..5 one query row per thread (TMEM lane quarter = warp mod 4); lane 0
//              of warp 2 issues the products: PV(j), then S(j + 1)
// TMEM (256 columns): S (then P, bf16) 0, O 128.
#include "internal.h"
#include "ptx.cuh"
#include "walk.cuh"

namespace ctxattn {
namespace {

template <int D>
struct WinLayout {
    static constexpr int NBOX = D / 64;
    static constexpr uint32_t BOX = kTile * 128;
    static constexpr uint32_t TILE = kTile * D * 2;
    // K(j + 1) is loaded while the softmax of tile j runs, V(j + 1) from PV(j)
    // on: one stage of each is what half an SM holds at D = 128
    static constexpr int STAGES = D == 64 ? 2 : 1;
    static constexpr uint32_t OFF_Q = 0;  // later the output's rows
    static constexpr uint32_t OFF_K = OFF_Q + TILE;
    static constexpr uint32_t OFF_V = OFF_K + STAGES * TILE;
    static constexpr uint32_t SMEM = OFF_V + STAGES * TILE + 1024;  // + alignment slack
    static constexpr uint32_t TM_S = 0, TM_O = 128, TM_COLS = 256;
};

struct WinBars {
    uint64_t q_full;
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_done, o_done, drain;
};

constexpr int kThreads = 192;
constexpr int kRowThreads = 128;
constexpr int kRowWarp0 = 2;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

__device__ __forceinline__ int pick3(int o, int s, int h, int b) {
    return o == 0 ? s : (o == 1 ? h : b);
}
__device__ __forceinline__ void tma_tile(const TmaMap& m, uint32_t dst, uint32_t bar, int d0, int s, int h, int b) {
    tma_load_4d(dst, &m.map, bar, d0, pick3(m.ord[0], s, h, b), pick3(m.ord[1], s, h, b), pick3(m.ord[2], s, h, b));
}
// Bounded wait that ignores the abort flag (teardown).
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > limit_ns) break;
}
// A bounded wait of a whole warp: one answer for all its lanes.  A lane whose
// wait runs out just as another's succeeds would otherwise leave the warp
// without it at the next warp-wide TMEM access, which then never completes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& w) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, w));
}

// The hand-over of P from the 128 row threads to the issuing warp: the others
// only arrive.  (An mbarrier with 128 arrivals in its place, and a walk
// state four registers larger: 633 instead of 522 us at S = 32760, 24 heads,
// D = 128, window 1024, when tiles still ended with the eight chunks; 509 now,
// 800 TFLOP/s over the visible pairs.)
__device__ __forceinline__ void rows_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kRowThreads) : "memory");
}
__device__ __forceinline__ void rows_arrive() {
    asm volatile("bar.arrive 1, %0;" ::"n"(kRowThreads) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) attn_window_kernel(const __grid_constant__ FwdParams p) {
    griddep_wait();  // the previous kernel in the stream is complete (launch_kernel)
    griddep_launch_dependents();
    using L = WinLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ WinBars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    const uint32_t sbase = smem_u32(smem_raw) + pad;
    const uint32_t sQ = sbase + L::OFF_Q, sK = sbase + L::OFF_K, sV = sbase + L::OFF_V;
    const int warp = warp_id(), lane = lane_id();
    const ChunkTable& ct = p.ct;
    const int tq = ct.ntiles - 1 - (int)blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int r = chunk_of_tile(ct, tq);
    const int q_start = ct.off[r] + (tq - ct.tile_off[r]) * kTile;
    const int q_rows = min(kTile, ct.off[r + 1] - q_start);
    const int hk = h / p.group;
    const WinKv wk = win_kv(ct, p.win, p.S, q_start, q_start + q_rows - 1);
    const int n_kv = wk.count();
    const WaitCtx wc{&abort_flag, p.status, p.timeout_ns};

    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(smem_u32(&bars.q_full), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.k_full[i]), 1);
            mbar_init(smem_u32(&bars.k_empty[i]), 1);
            mbar_init(smem_u32(&bars.v_full[i]), 1);
            mbar_init(smem_u32(&bars.v_empty[i]), 1);
        }
        mbar_init(smem_u32(&bars.s_done), 1);
        mbar_init(smem_u32(&bars.o_done), 1);
        mbar_init(smem_u32(&bars.drain), 1);
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), L::TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    auto stage_of = [](int j) { return j % L::STAGES; };
    auto phase_of = [](int j) { return (j / L::STAGES) & 1; };

    if (warp < kRowWarp0) {
        // ------------------------------------------------------ TMA producers
        // Two loading threads, Q and K from warp 0 and V from warp 1: one
        // thread's copies stream at about 35 B per clock, a third of a step's
        // time for the K and V tiles together.
        if (lane == 0) {
            const bool isv = warp == 1;
            const uint32_t qf = smem_u32(&bars.q_full), sT = isv ? sV : sK;
            const TmaMap& map = isv ? p.tv : p.tk;
            uint64_t* full = isv ? bars.v_full : bars.k_full;
            uint64_t* empty = isv ? bars.v_empty : bars.k_empty;
            if (!isv) {
                mbar_arrive_expect_tx(qf, L::TILE);
                for (int bx = 0; bx < L::NBOX; ++bx)
                    tma_tile(p.tq, sQ + bx * L::BOX, qf, bx * 64, q_start, h, b);
            }
            int last[2] = {-1, -1};
            bool ok = true;
            const int skip = debug_skip_step(p.debug, n_kv);  // -1 in normal use
            KvWalk w;
            win_first(ct, wk, w);
            for (int j = 0; j < n_kv; ++j, win_next(ct, wk, w)) {
                if (j == skip) {  // failure injection: no K, V from step j on
                    ok = false;
                    break;
                }
                const int st = stage_of(j), ph = phase_of(j);
                const int kv_start = ct.off[w.c] + (w.t - w.t0) * kTile;
                if (!(ok = mbar_wait(smem_u32(&empty[st]), ph ^ 1, wc))) break;
                const uint32_t f = smem_u32(&full[st]);
                mbar_arrive_expect_tx(f, L::TILE);
                for (int bx = 0; bx < L::NBOX; ++bx)
                    tma_tile(map, sT + st * L::TILE + bx * L::BOX, f, bx * 64, kv_start, hk, b);
                last[st] = ph;
            }
            if (!ok) {
                // wait for our own copies in flight before the CTA retires
                if (!isv) drain_wait(qf, 0, p.timeout_ns);
                for (int st = 0; st < 2; ++st)
                    if (last[st] >= 0) drain_wait(smem_u32(&full[st]), last[st], p.timeout_ns);
            }
        }
    } else if (warp >= kRowWarp0) {
        // ------------------------------------------------------ softmax + MMA issue
        const int quarter = warp & 3;  // the TMEM lanes this warp may read
        const int row = quarter * 32 + lane;
        const bool issuer = warp == kRowWarp0 && lane == 0;
        const uint32_t taddr = tmem + (uint32_t(quarter * 32) << 16);
        const float sc = p.scale_log2;
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, false, true);
        const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024), dk0 = sdesc_sw128(sK, 16, 1024);
        const uint64_t dv0 = sdesc_sw128(sV, L::BOX, 1024);
        const uint32_t s_done = smem_u32(&bars.s_done);
        auto issue_s = [&](int j) {  // S = Q K^T
            const int st = stage_of(j);
            const uint64_t bk = dk0 + ((st * L::TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t koff = ((kk >> 2) * L::BOX + (kk & 3) * 32) >> 4;
                mma_ss(tmem + L::TM_S, dq0 + koff, bk + koff, idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit(s_done);
            mma_commit(smem_u32(&bars.k_empty[st]));
        };
        bool ok = true;
        if (issuer) {
            ok = mbar_wait(smem_u32(&bars.q_full), 0, wc) && mbar_wait(smem_u32(&bars.k_full[0]), 0, wc);
            if (ok) issue_s(0);
            else *wc.abort_flag = 1;
        }
        ok = __all_sync(0xffffffffu, ok);
        float m_ref = -INFINITY, l = 0.f;
        int c = 0;
        for (int j = 0; j < n_kv && ok; ++j) {
            const int t = win_tile(wk, j);
            c = win_chunk(ct, t, c);
            const int kv_start = ct.off[c] + (t - ct.tile_off[c]) * kTile;
            const int kv_len = min(kTile, ct.off[c + 1] - kv_start);
            if (!(ok = warp_wait(s_done, j & 1, wc))) {
                if (warp != kRowWarp0) rows_arrive();  // so that the issuing warp does not wait for this one
                break;
            }
            tc_fence_after();
            uint32_t s[128];
            tmem_ld128_sync(taddr + L::TM_S, s);
            mask_window(p.win, q_start, row, kv_start, kv_len, s);
            float mx8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) mx8[e] = __uint_as_float(s[e]);
#pragma unroll
            for (int k = 8; k < 128; k += 8)
#pragma unroll
                for (int e = 0; e < 8; ++e) mx8[e] = fmaxf(mx8[e], __uint_as_float(s[k + e]));
            const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                   fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
            float alpha = 1.f;
            bool rescale = false;
            if (mx > m_ref) {
                if (m_ref == -INFINITY) {
                    m_ref = mx;  // nothing accumulated yet for this row
                } else if ((mx - m_ref) * sc > kRescaleThreshold) {
                    alpha = ex2((m_ref - mx) * sc);
                    m_ref = mx;
                    rescale = true;
                }
            }
            const float neg = m_ref == -INFINITY ? 0.f : -m_ref * sc;  // a row with no key yet
            float sum8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 64; ++k) {
                float x0, x1;
                if constexpr (D == 64) {  // two-lane instructions, as in attn_fwd.cu
                    const float2 v = ffma2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])),
                                           make_float2(sc, sc), make_float2(neg, neg));
                    x0 = v.x;
                    x1 = v.y;
                } else {
                    x0 = fmaf(__uint_as_float(s[2 * k]), sc, neg);
                    x1 = fmaf(__uint_as_float(s[2 * k + 1]), sc, neg);
                }
                const float p0 = ex2(x0), p1 = ex2(x1);
                sum8[(2 * k) & 7] += p0;
                sum8[(2 * k + 1) & 7] += p1;
                s[k] = pack_bf16x2(p0, p1);  // packed P overwrites scores already consumed
            }
            tmem_st32(taddr + L::TM_S + 0, s);
            tmem_st32(taddr + L::TM_S + 32, s + 32);
            l = l * alpha + (((sum8[0] + sum8[1]) + (sum8[2] + sum8[3])) + ((sum8[4] + sum8[5]) + (sum8[6] + sum8[7])));
            if (__any_sync(0xffffffffu, rescale)) {
                // PV(j - 1) was issued before S(j) by the same thread and has
                // completed with it: rescale O in place
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    tmem_ld32_sync(taddr + L::TM_O + cc * 32, o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                    tmem_st32(taddr + L::TM_O + cc * 32, o);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            // Every row's P (and O rescale) is in TMEM.  Only the issuing warp
            // waits; a warp that has given up has raised the abort flag first.
            if (warp != kRowWarp0) {
                rows_arrive();
                continue;
            }
            rows_sync();
            ok = *wc.abort_flag == 0;
            if (issuer && ok) {
                const int st = stage_of(j);
                ok = mbar_wait(smem_u32(&bars.v_full[st]), phase_of(j), wc);
                tc_fence_after();
                if (ok) {
                    const uint64_t bv = dv0 + ((st * L::TILE) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_ts(tmem + L::TM_O, tmem + L::TM_S + kk * 8, bv + kk * (2048 >> 4), idesc_pv,
                               (j > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(smem_u32(&bars.v_empty[st]));
                    if (j + 1 == n_kv) {
                        mma_commit(smem_u32(&bars.o_done));
                    } else {
                        // S(j + 1) overwrites P(j): behind the PV that reads it (in order)
                        ok = mbar_wait(smem_u32(&bars.k_full[stage_of(j + 1)]), phase_of(j + 1), wc);
                        if (ok) issue_s(j + 1);
                    }
                }
                if (!ok) *wc.abort_flag = 1;
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        // --------------------------------------------------------- epilogue
        if (ok && warp_wait(smem_u32(&bars.o_done), 0, wc)) {
            tc_fence_after();
            const float inv_l = 1.f / l;
            // Rows go out through the memory Q was in (its last product is done):
            // 64 columns at a time a warp stores its 32 rows swizzled and reads
            // them back eight lanes to a row, so that global stores are whole
            // 128-byte lines instead of 16 bytes in each of 32 rows.
            const uint32_t stage = sQ + quarter * 4096;
            __nv_bfloat16* out = p.out + (int64_t)b * p.o_sb + (int64_t)(q_start + quarter * 32) * p.o_ss + (int64_t)h * p.o_sh;
#pragma unroll
            for (int hc = 0; hc < D / 64; ++hc) {
                uint32_t o[64];
                tmem_ld64_sync(taddr + L::TM_O + hc * 64, o);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + sw128_offset(lane, k)),
                                 "r"(pack_bf16x2(__uint_as_float(o[8 * k + 0]) * inv_l, __uint_as_float(o[8 * k + 1]) * inv_l)),
                                 "r"(pack_bf16x2(__uint_as_float(o[8 * k + 2]) * inv_l, __uint_as_float(o[8 * k + 3]) * inv_l)),
                                 "r"(pack_bf16x2(__uint_as_float(o[8 * k + 4]) * inv_l, __uint_as_float(o[8 * k + 5]) * inv_l)),
                                 "r"(pack_bf16x2(__uint_as_float(o[8 * k + 6]) * inv_l, __uint_as_float(o[8 * k + 7]) * inv_l))
                                 : "memory");
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int rr = 4 * k + (lane >> 3);
                    uint4 v;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(stage + sw128_offset(rr, lane & 7)) : "memory");
                    if (quarter * 32 + rr < q_rows)
                        *reinterpret_cast<uint4*>(out + (int64_t)rr * p.o_ss + hc * 64 + (lane & 7) * 8) = v;
                }
                __syncwarp();
            }
            if (row < q_rows) p.lse[((int64_t)b * p.Hq + h) * p.S + q_start + row] = m_ref * p.scale + logf(l);
        }
    }

    if (warp == kRowWarp0 && lane == 0) {
        mma_commit(smem_u32(&bars.drain));  // this CTA's products must retire first
        drain_wait(smem_u32(&bars.drain), 0, p.timeout_ns);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, L::TM_COLS);
}

template <int D>
int launch_window_d(const FwdParams& p, cudaStream_t s) {
    using L = WinLayout<D>;
    static OncePerDevice attr;
    if (!attr.run([] {
            return cudaFuncSetAttribute(attn_window_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM) ==
                   cudaSuccess;
        }))
        return 4;
    const cudaError_t e = launch_kernel(p.pdl != 0, attn_window_kernel<D>, dim3(p.ct.ntiles, p.Hq, p.B), dim3(kThreads),
                                        L::SMEM, s, p);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 0 : 4;
}

}  // namespace

int launch_attn_window_fwd(const FwdParams& p, int D, cudaStream_t s) {
    if (D == 64) return launch_window_d<64>(p, s);
    if (D == 128) return launch_window_d<128>(p, s);
    return launch_attn_fwd256(p, s);
}

}  // namespace ctxattn

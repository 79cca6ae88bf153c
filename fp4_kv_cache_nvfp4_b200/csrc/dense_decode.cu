// Dense decode attention: one token per sequence over every entry of the FP4
// main KV.
//
// Mathematics.  One pass over the entries with a running maximum m and sum l per
// head (log2 domain): p_j = 2^(s_j - m), l = sum p_j, O = sum p_j v_j; parts of
// a sequence are joined by rescaling with 2^(m_part - m).  m follows the scores
// lazily: it is raised only when a score exceeds it by more than 2^8, so O is
// rescaled a few times per sequence.  p carries a factor of 2^7 (at most 2^15
// as fp16), which keeps weights down to 2^-21 of the largest at fp16's full precision.
//
// What bounds it.  144 bytes per entry for 8192 FLOP (16 heads share K and V):
// HBM, if dequantisation and mma.sync stay behind the copies.  So
//   * the entries of all sequences form one list of 128-entry tiles, of which
//     every CTA (one per SM) takes an equal contiguous share, whatever the
//     lengths; a sequence that spans CTAs leaves partial results that a second
//     kernel joins;
//   * one warp copies tiles into a ring with TMA (codes as 128-byte-swizzled
//     boxes of at most a page, scales as one bulk copy per box);
//   * each of eight warps takes 16 entries of a tile, dequantises them in
//     registers straight into mma.sync fragments (E2M1 x E4M3 is exact in fp16)
//     and keeps its own m, l and O, joined once per sequence.  Nothing is
//     written back to shared memory on the way.
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace csa2 {

constexpr int DD_WARPS = 8;                     // consumer warps, 16 entries of a tile each
constexpr int DD_TILE = 16 * DD_WARPS;          // entries per tile
constexpr int DD_STAGES = 7;
constexpr int DD_THREADS = (DD_WARPS + 1) * 32;
constexpr int DD_CODES = DD_TILE * kCodeBytes;  // 16 KiB per stage
constexpr int DD_SCALES = DD_TILE * kScales;    // 2 KiB
constexpr int DD_OROW = kD + 4;                 // floats per row of the joining slab (bank spread)
constexpr size_t DD_OFF_CODES = 0;
constexpr size_t DD_OFF_SCALES = DD_OFF_CODES + (size_t)DD_STAGES * DD_CODES;
constexpr size_t DD_OFF_SLAB = DD_OFF_SCALES + (size_t)DD_STAGES * DD_SCALES;  // [warps][16][DD_OROW] floats
constexpr size_t DD_OFF_M = DD_OFF_SLAB + (size_t)DD_WARPS * kH * DD_OROW * 4;  // [warps][16]
constexpr size_t DD_OFF_L = DD_OFF_M + DD_WARPS * kH * 4;                      // [warps][16]
constexpr size_t DD_OFF_OK = DD_OFF_L + DD_WARPS * kH * 4;                     // [stages][16] bytes: boxes of 8 entries present
constexpr size_t DD_OFF_BAR = DD_OFF_OK + DD_STAGES * 16;
constexpr size_t DD_OFF_MISC = DD_OFF_BAR + 2 * DD_STAGES * 8;
constexpr size_t DD_SMEM = DD_OFF_MISC + 64;
static_assert(DD_OFF_SCALES % 16 == 0 && DD_OFF_SLAB % 16 == 0 && DD_OFF_OK % 16 == 0 && DD_OFF_BAR % 8 == 0,
              "dense decode layout");
static_assert(DD_SMEM <= 227 * 1024, "dense decode shared memory");

struct DecodeArgs {
    DenseArgs a;
    float* part_o;  // [2 * ctas][16][128], times 2^(kPBias - m)
    float* part_m;  // [2 * ctas][16] maxima (log2 domain)
    float* part_l;  // [2 * ctas][16] sums
    int4* cut;      // [ctas]: (sequence, its first tile, its end, first tile of this CTA) if it begins inside one
};

// ---- which tiles ----------------------------------------------------------------
// Sequence b's length, 0 if it is out of range.
__device__ __forceinline__ int dense_len(const DenseArgs& a, int b) {
    const int n = __ldg(a.seq_lens + b);
    return n < 0 || n > a.max_len ? 0 : n;
}

// One tile's address of an entry row's 16-byte chunk c (0..7) of the swizzled codes
__device__ __forceinline__ uint32_t dd_chunk(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

template <bool SPLIT>
__global__ void __launch_bounds__(DD_THREADS, 1)
    dense_decode_kernel(const __grid_constant__ CUtensorMap map, const DecodeArgs d) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const DenseArgs& a = d.a;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + DD_OFF_BAR);
    uint64_t* empty = full + DD_STAGES;
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + DD_OFF_MISC);
    volatile uint32_t* s_timeout = misc;  // [0]; [1..3]: start sequence, its first tile, total
    uint8_t* s_ok = smem + DD_OFF_OK;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(smem) & 1023u) {  // uniform over the grid
        pdl_wait();
        if (tid == 0) dev_error(a.err, CSA2_DEV_ALIGN);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < DD_STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], DD_WARPS);
        }
        *s_timeout = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share of the tiles: [lo, hi) of the flattened list ------------
    uint32_t* scan = reinterpret_cast<uint32_t*>(smem + DD_OFF_SLAB);
    const int per_thread = (a.B + DD_THREADS - 1) / DD_THREADS;
    const int b0 = min(a.B, tid * per_thread), b1 = min(a.B, b0 + per_thread);
    uint32_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        mine += (uint32_t)(dense_len(a, b) + DD_TILE - 1) / DD_TILE;
        if (blockIdx.x == 0) {
            const int n = __ldg(a.seq_lens + b);
            if (n < 0 || n > a.max_len) dev_error(a.err, CSA2_DEV_LEN);
        }
    }
    uint32_t total;
    const uint32_t before = block_excl_scan(mine, scan, &total);
    const uint32_t per = (total + gridDim.x - 1) / gridDim.x;
    const uint32_t lo = min(total, per * blockIdx.x), hi = min(total, lo + per);
    if (lo >= before && lo < before + mine) {
        uint32_t t = before;
        for (int b = b0; b < b1; ++b) {
            const uint32_t n = (uint32_t)(dense_len(a, b) + DD_TILE - 1) / DD_TILE;
            if (lo < t + n) {
                misc[1] = (uint32_t)b;
                misc[2] = t;
                break;
            }
            t += n;
        }
    }
    __syncthreads();
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // bounded; after one timeout every wait returns at once
        if (*s_timeout) return;
        if (!mbar_wait(bar, parity, kDenseWaitLimit)) *s_timeout = 1;
    };
    const int sh = a.page_shift;

    if (lo < hi && warp == DD_WARPS) {
        // ================= copies: one lane per box (at most a page) =================
        const int box_shift = min(sh, 7), box = 1 << box_shift, n_box = DD_TILE >> box_shift;
        int b = (int)misc[1];
        uint32_t t0 = misc[2];
        int n = dense_len(a, b);
        uint32_t t1 = t0 + (uint32_t)(n + DD_TILE - 1) / DD_TILE;
        // entry position and page (not checked yet) of this lane's box of tile t; -1: no box
        auto seek = [&](uint32_t t, int& pos, int32_t& pg) {
            while (t >= t1) {  // the next sequence that has tiles
                n = dense_len(a, ++b);
                t0 = t1;
                t1 += (uint32_t)(n + DD_TILE - 1) / DD_TILE;
            }
            pos = (int)(t - t0) * DD_TILE + lane * box;
            pg = -1;
            if (lane >= n_box || pos >= n) pos = -1;
            else pg = __ldg(a.cache.page_table + (int64_t)b * a.cache.max_pages_per_seq + (pos >> sh));
        };
        uint32_t done = 0;
        int pos_next;
        int32_t pg_next;
        seek(lo, pos_next, pg_next);
        for (uint32_t t = lo; t < hi; ++t, ++done) {
            const int pos = pos_next;
            int32_t pg = pg_next;
            if (pos >= 0 && (pg < 0 || pg >= a.cache.n_phys_pages)) {
                dev_error(a.err, CSA2_DEV_PAGE);
                pg = -1;
            }
            if (t + 1 < hi) seek(t + 1, pos_next, pg_next);  // in flight while this tile waits for its stage
            const int s = (int)(done % DD_STAGES);
            if (done >= DD_STAGES) wait(&empty[s], (done / DD_STAGES - 1) & 1u);
            if (*s_timeout) break;
            if (lane < n_box)  // eight entries per flag
                for (int k = 0; k < box / 8; ++k) s_ok[s * 16 + lane * (box / 8) + k] = pg >= 0;
            const int boxes = __popc(__ballot_sync(0xffffffffu, pg >= 0));
            if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)boxes * (uint32_t)box * (kCodeBytes + kScales));
            __syncwarp();
            if (pg >= 0) {
                const int slot = (pg << sh) | (pos & ((1 << sh) - 1));
                tma_load_2d(smem + DD_OFF_CODES + (size_t)s * DD_CODES + (size_t)lane * box * kCodeBytes, &map, 0, slot,
                            &full[s]);
                bulk_load(smem + DD_OFF_SCALES + (size_t)s * DD_SCALES + (size_t)lane * box * kScales,
                          a.cache.scales + (int64_t)slot * kScales, (uint32_t)box * kScales, &full[s]);
            }
            __syncwarp();
        }
        // no copy is in flight when the CTA ends, whoever gave up
        if (*s_timeout)
            for (uint32_t k = done > DD_STAGES ? done - DD_STAGES : 0; k < done; ++k)
                mbar_wait(&full[k % DD_STAGES], (k / DD_STAGES) & 1u, kDenseWaitLimit);
    } else if (lo < hi) {
        // ================= eight consumer warps =================
        const int g = lane >> 2, t4 = lane & 3;
        // Fragment column g (and columns 2 t, 2 t + 1) of an 8-entry group is entry
        // perm(g): its order keeps the swizzled reads of K (16 bytes, lanes g, t)
        // and V (8 bytes, the columns' entries) free of bank conflicts.
        const int kg = ((g >> 1) ^ (((g >> 1) & 1) << 2)) ^ ((g & 1) << 2);
        const int va = t4 ^ ((t4 & 1) << 2), vb = va ^ 4;
        const GroupBar bar{1, DD_WARPS * 32};
        float* slab = reinterpret_cast<float*>(smem + DD_OFF_SLAB);
        float* wm = reinterpret_cast<float*>(smem + DD_OFF_M);
        float* wl = reinterpret_cast<float*>(smem + DD_OFF_L);
        int b = (int)misc[1];
        uint32_t t0 = misc[2];
        int n = dense_len(a, b);
        uint32_t t1 = t0 + (uint32_t)(n + DD_TILE - 1) / DD_TILE;
        if (tid == 0) d.cut[blockIdx.x] = lo > t0 ? make_int4(b, (int)t0, (int)t1, (int)lo) : make_int4(-1, 0, 0, 0);
        uint32_t t = lo, done = 0;
        while (t < hi) {
            while (t >= t1) {
                n = dense_len(a, ++b);
                t0 = t1;
                t1 += (uint32_t)(n + DD_TILE - 1) / DD_TILE;
            }
            const uint32_t seg0 = t, seg1 = min(hi, t1);
            // ---- Q of the sequence: heads g and g + 8, channels 32 t .. 32 t + 31 -------
            uint32_t qa[8][4];
            float c0, c1;  // score (log2 domain) = product * c
            {
                const uint4* qg = reinterpret_cast<const uint4*>(a.q + ((int64_t)b * kH + g) * kD + 32 * t4);
                uint4 r0[4], r1[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r0[i] = __ldg(qg + i);
                    r1[i] = __ldg(qg + 8 * kD / 8 + i);
                }
                float f0, f1;
                q_scale(quad_max(q_absmax(r0)), f0, c0);
                q_scale(quad_max(q_absmax(r1)), f1, c1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qa[2 * i][0] = q_half2(r0[i].x, f0);
                    qa[2 * i][1] = q_half2(r1[i].x, f1);
                    qa[2 * i][2] = q_half2(r0[i].y, f0);
                    qa[2 * i][3] = q_half2(r1[i].y, f1);
                    qa[2 * i + 1][0] = q_half2(r0[i].z, f0);
                    qa[2 * i + 1][1] = q_half2(r1[i].z, f1);
                    qa[2 * i + 1][2] = q_half2(r0[i].w, f0);
                    qa[2 * i + 1][3] = q_half2(r1[i].w, f1);
                }
            }
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
            float bias0 = kPBias, bias1 = kPBias;  // kPBias - m
            float O[16][4];
#pragma unroll
            for (int i = 0; i < 16; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.f;

            for (; t < seg1; ++t, ++done) {
                const int s = (int)(done % DD_STAGES);
                wait(&full[s], (done / DD_STAGES) & 1u);
                const int u0 = (int)(t - t0) * DD_TILE + 16 * warp;  // first entry of this warp's unit
                if (u0 >= n) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[s]);
                    continue;
                }
                const uint8_t* codes = smem + DD_OFF_CODES + (size_t)s * DD_CODES + (size_t)warp * 16 * kCodeBytes;
                const uint8_t* scales = smem + DD_OFF_SCALES + (size_t)s * DD_SCALES + (size_t)warp * 16 * kScales;
                const uint32_t ok2 = *reinterpret_cast<const uint16_t*>(s_ok + s * 16 + 2 * warp);
                uint4 kc[2];
                uint32_t ks[2];
                uint2 vc[2][2];
                uint32_t vs[2];  // (scale of entry va, scale of entry vb) as two bytes
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    kc[j] = *reinterpret_cast<const uint4*>(codes + dd_chunk(8 * j + kg, t4));
                    ks[j] = *reinterpret_cast<const uint16_t*>(scales + (8 * j + kg) * kScales + 2 * t4);
                    vc[j][0] = *reinterpret_cast<const uint2*>(codes + dd_chunk(8 * j + va, 4 + (g >> 1)) + 8 * (g & 1));
                    vc[j][1] = *reinterpret_cast<const uint2*>(codes + dd_chunk(8 * j + vb, 4 + (g >> 1)) + 8 * (g & 1));
                    vs[j] = (uint32_t)scales[(8 * j + va) * kScales + 8 + g] |
                            ((uint32_t)scales[(8 * j + vb) * kScales + 8 + g] << 8);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);  // everything of the unit is in registers
                // entries behind the last one, or of a missing page: scale 0, score -inf
                const bool whole = ok2 == 0x0101u && u0 + 16 <= n;
                bool seen[2][2] = {{true, true}, {true, true}};
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const bool box_ok = (ok2 >> (8 * j)) & 1u;
                        if (!box_ok || u0 + 8 * j + kg >= n) ks[j] = 0;
                        seen[j][0] = box_ok && u0 + 8 * j + va < n;
                        seen[j][1] = box_ok && u0 + 8 * j + vb < n;
                        if (!seen[j][0]) vs[j] &= 0xff00u;
                        if (!seen[j][1]) vs[j] &= 0x00ffu;
                    }
                }
                // ---- S = Q K^T -------------------------------------------------------------
                float S[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                uint32_t kl[2], kh[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t s2 = e4m3x2_to_h2(ks[j]);
                    kl[j] = __byte_perm(s2, 0u, 0x1010);
                    kh[j] = __byte_perm(s2, 0u, 0x3232);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t w = i == 0 ? kc[j].x : i == 1 ? kc[j].y : i == 2 ? kc[j].z : kc[j].w;
                        const uint32_t sc = i < 2 ? kl[j] : kh[j];
                        uint32_t h0, h1, h2, h3;
                        e2m1x8_to_h2x4(w, h0, h1, h2, h3);
                        mma16816(S[j], qa[2 * i], hmul2(h0, sc), hmul2(h1, sc));
                        mma16816(S[j], qa[2 * i + 1], hmul2(h2, sc), hmul2(h3, sc));
                    }
                }
                // ---- weights ---------------------------------------------------------------
                float x[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    x[j][0] = fmaf(S[j][0], c0, bias0);
                    x[j][1] = fmaf(S[j][1], c0, bias0);
                    x[j][2] = fmaf(S[j][2], c1, bias1);
                    x[j][3] = fmaf(S[j][3], c1, bias1);
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!seen[j][e]) x[j][e] = x[j][2 + e] = -INFINITY;
                    }
                }
                float mx0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
                float mx1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
                const bool rise = mx0 > kPMax || mx1 > kPMax || m0 == -INFINITY || m1 == -INFINITY;
                if (__any_sync(0xffffffffu, rise)) {
                    mx0 = quad_max(mx0) - bias0;  // the scores' maxima
                    mx1 = quad_max(mx1) - bias1;
                    const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
                    const float nb0 = n0 == -INFINITY ? kPBias : kPBias - n0, nb1 = n1 == -INFINITY ? kPBias : kPBias - n1;
                    const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        x[j][0] += nb0 - bias0;
                        x[j][1] += nb0 - bias0;
                        x[j][2] += nb1 - bias1;
                        x[j][3] += nb1 - bias1;
                    }
                    m0 = n0, m1 = n1, bias0 = nb0, bias1 = nb1;
                    l0 *= f0, l1 *= f1;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        O[i][0] *= f0;
                        O[i][1] *= f0;
                        O[i][2] *= f1;
                        O[i][3] *= f1;
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[j][e] = ex2(x[j][e]);
                    l0 += x[j][0] + x[j][1];
                    l1 += x[j][2] + x[j][3];
                }
                const uint32_t pa[4] = {f2_to_h2(x[0][0], x[0][1]), f2_to_h2(x[0][2], x[0][3]),
                                        f2_to_h2(x[1][0], x[1][1]), f2_to_h2(x[1][2], x[1][3])};
                uint32_t pl[4];
                if (SPLIT) {  // what the first fp16 term leaves
                    pl[0] = rest_h2(x[0][0], x[0][1], pa[0]);
                    pl[1] = rest_h2(x[0][2], x[0][3], pa[1]);
                    pl[2] = rest_h2(x[1][0], x[1][1], pa[2]);
                    pl[3] = rest_h2(x[1][2], x[1][3], pa[3]);
                }
                // ---- O += P V: tile i of eight columns is dims 16 g + i --------------------
                const uint32_t sc0 = e4m3x2_to_h2(vs[0]), sc1 = e4m3x2_to_h2(vs[1]);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    // nibble pairs (entry va, entry vb) of one dim in one byte: even dims, then odd dims
                    uint32_t ev[2], od[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t p = w ? vc[j][0].y : vc[j][0].x, q = w ? vc[j][1].y : vc[j][1].x;
                        ev[j] = (p & 0x0f0f0f0fu) | ((q << 4) & 0xf0f0f0f0u);
                        od[j] = ((p >> 4) & 0x0f0f0f0fu) | (q & 0xf0f0f0f0u);
                    }
                    uint32_t e0[4], e1[4], o0[4], o1[4];
                    e2m1x8_to_h2x4(ev[0], e0[0], e0[1], e0[2], e0[3]);
                    e2m1x8_to_h2x4(ev[1], e1[0], e1[1], e1[2], e1[3]);
                    e2m1x8_to_h2x4(od[0], o0[0], o0[1], o0[2], o0[3]);
                    e2m1x8_to_h2x4(od[1], o1[0], o1[1], o1[2], o1[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x0 = hmul2(e0[i], sc0), x1 = hmul2(e1[i], sc1);
                        const uint32_t y0 = hmul2(o0[i], sc0), y1 = hmul2(o1[i], sc1);
                        mma16816(O[8 * w + 2 * i], pa, x0, x1);
                        mma16816(O[8 * w + 2 * i + 1], pa, y0, y1);
                        if (SPLIT) {
                            mma16816(O[8 * w + 2 * i], pl, x0, x1);
                            mma16816(O[8 * w + 2 * i + 1], pl, y0, y1);
                        }
                    }
                }
            }

            // ---- join the eight warps' results of the segment ------------------------------
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            if (t4 == 0) {
                wm[warp * kH + g] = m0;
                wm[warp * kH + g + 8] = m1;
                wl[warp * kH + g] = l0;
                wl[warp * kH + g + 8] = l1;
            }
            bar.sync();
            float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
            for (int w = 0; w < DD_WARPS; ++w) {
                M0 = fmaxf(M0, wm[w * kH + g]);
                M1 = fmaxf(M1, wm[w * kH + g + 8]);
            }
            const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M1);
            // columns 2 t and 2 t + 1 of tile i are dims 32 t + i and 32 t + 16 + i
            float* my = slab + ((size_t)warp * kH + g) * DD_OROW + 32 * t4;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                *reinterpret_cast<float4*>(my + i) =
                    make_float4(O[i][0] * f0, O[i + 1][0] * f0, O[i + 2][0] * f0, O[i + 3][0] * f0);
                *reinterpret_cast<float4*>(my + 16 + i) =
                    make_float4(O[i][1] * f0, O[i + 1][1] * f0, O[i + 2][1] * f0, O[i + 3][1] * f0);
                *reinterpret_cast<float4*>(my + 8 * DD_OROW + i) =
                    make_float4(O[i][2] * f1, O[i + 1][2] * f1, O[i + 2][2] * f1, O[i + 3][2] * f1);
                *reinterpret_cast<float4*>(my + 8 * DD_OROW + 16 + i) =
                    make_float4(O[i][3] * f1, O[i + 1][3] * f1, O[i + 2][3] * f1, O[i + 3][3] * f1);
            }
            bar.sync();
            {
                const int h = tid >> 4, d8 = (tid & 15) * 8;  // 16 heads x 16 threads of 8 dims
                float M = -INFINITY, l = 0.f, o[8];
#pragma unroll
                for (int w = 0; w < DD_WARPS; ++w) M = fmaxf(M, wm[w * kH + h]);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll
                for (int w = 0; w < DD_WARPS; ++w) {
                    const float mw = wm[w * kH + h];
                    if (mw != -INFINITY) l += wl[w * kH + h] * ex2(mw - M);
                    const float* p = slab + ((size_t)w * kH + h) * DD_OROW + d8;
                    const float4 v0 = *reinterpret_cast<const float4*>(p), v1 = *reinterpret_cast<const float4*>(p + 4);
                    o[0] += v0.x, o[1] += v0.y, o[2] += v0.z, o[3] += v0.w;
                    o[4] += v1.x, o[5] += v1.y, o[6] += v1.z, o[7] += v1.w;
                }
                if (seg0 == t0 && seg1 == t1) {  // the whole sequence
                    dense_store(a, (int64_t)b * kH + h, d8, o, M, l);
                } else {
                    const int64_t part = 2 * (int64_t)blockIdx.x + (seg0 == t0 ? 1 : 0);
                    float* po = d.part_o + (part * kH + h) * kD + d8;
                    *reinterpret_cast<float4*>(po) = make_float4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<float4*>(po + 4) = make_float4(o[4], o[5], o[6], o[7]);
                    if (d8 == 0) {
                        d.part_m[part * kH + h] = M;
                        d.part_l[part * kH + h] = l;
                    }
                }
            }
            bar.sync();  // the slab is free for the next segment
        }
    } else if (tid == 0) {
        d.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    // sequences without entries
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
        if (warp < DD_WARPS && dense_len(a, b) == 0) {
            const float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            dense_store(a, (int64_t)b * kH + (tid >> 4), (tid & 15) * 8, o, -INFINITY, 0.f);
        }
    __syncthreads();
    if (tid == 0 && *s_timeout) dev_error(a.err, CSA2_DEV_TIMEOUT);
}

// Joins the partial results of every sequence that spans CTAs: block (c, y) the
// heads 4 y .. 4 y + 3 of the sequence that CTA c continues, if CTA c - 1 began
// it.  Four warps per head share the parts; sums in a fixed order.
constexpr int DJ_THREADS = 512;
__global__ void __launch_bounds__(DJ_THREADS) dense_decode_join_kernel(const DecodeArgs d) {
    __shared__ float4 s_o[16][32];
    __shared__ float s_l[16];
    const DenseArgs& a = d.a;
    const int c = blockIdx.x + 1, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_trigger();
    const int4 cut = d.cut[c];
    if (cut.x < 0) return;
    const int per = cut.w / c;  // CTA c begins at tile c * per
    if (cut.y < (c - 1) * per) return;  // an earlier CTA's block does it
    const int last = (cut.z - 1) / per, n = last - c + 2;
    const int h = 4 * blockIdx.y + (warp >> 2), w4 = warp & 3;
    auto part = [&](int k) { return (int64_t)(k == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + k)) * kH + h; };
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, d.part_m[part(k)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 8
    for (int k = w4; k < n; k += 4) {
        const int64_t p = part(k);
        const float m = d.part_m[p];
        const float4 v = *reinterpret_cast<const float4*>(d.part_o + p * kD + 4 * lane);
        const float f = m == -INFINITY ? 0.f : ex2(m - M);
        o.x += v.x * f;
        o.y += v.y * f;
        o.z += v.z * f;
        o.w += v.w * f;
        l += d.part_l[p] * f;
    }
    s_o[warp][lane] = o;
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (w4 == 0 && lane < 16) {
        float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        l = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float4 x = s_o[warp + w][2 * lane], y = s_o[warp + w][2 * lane + 1];
            r[0] += x.x, r[1] += x.y, r[2] += x.z, r[3] += x.w;
            r[4] += y.x, r[5] += y.y, r[6] += y.z, r[7] += y.w;
            l += s_l[warp + w];
        }
        dense_store(a, (int64_t)cut.x * kH + h, 8 * lane, r, M, l);
    }
}

size_t dense_decode_ws_bytes() {
    return (size_t)2 * kDenseCtas * kH * (kD + 2) * 4 + (size_t)kDenseCtas * sizeof(int4);
}

cudaError_t launch_dense_decode(const DenseArgs& a, char* ws, cudaStream_t stream) {
    static bool init[64];
    static int n_sm[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!init[dev]) {
        for (const void* k : {(const void*)dense_decode_kernel<false>, (const void*)dense_decode_kernel<true>}) {
            e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)DD_SMEM);
            if (e != cudaSuccess) return e;
        }
        e = cudaDeviceGetAttribute(&n_sm[dev], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        init[dev] = true;
    }
    CUtensorMap map;
    if (!dense_code_map(a.cache, &map, DD_TILE)) return cudaErrorInvalidValue;
    DecodeArgs d{};
    d.a = a;
    float* f = reinterpret_cast<float*>(ws);
    d.part_o = f;
    d.part_m = d.part_o + (size_t)2 * kDenseCtas * kH * kD;
    d.part_l = d.part_m + (size_t)2 * kDenseCtas * kH;
    d.cut = reinterpret_cast<int4*>(d.part_l + (size_t)2 * kDenseCtas * kH);
    const int64_t most = (int64_t)a.B * ((a.max_len + DD_TILE - 1) / DD_TILE);  // tiles there can be
    const unsigned ctas = (unsigned)std::min<int64_t>(std::min(n_sm[dev], kDenseCtas), most);
    LaunchCfg c(dim3(ctas), dim3(DD_THREADS), DD_SMEM, stream);
    e = a.out_bf16 ? cudaLaunchKernelEx(&c.cfg, dense_decode_kernel<false>, (const CUtensorMap)map, d)
                   : cudaLaunchKernelEx(&c.cfg, dense_decode_kernel<true>, (const CUtensorMap)map, d);
    if (e != cudaSuccess || ctas == 1) return e;
    LaunchCfg j(dim3(ctas - 1, kH / 4), dim3(DJ_THREADS), 0, stream);
    return cudaLaunchKernelEx(&j.cfg, dense_decode_join_kernel, d);
}

}  // namespace csa2

// Dense decode attention: one token per sequence over every entry of the FP4
// main KV.
//
// Mathematics.  One pass over the entries with a running maximum m and sum l per
// head (log2 domain): p_j = 2^(s_j - m), l = sum p_j, O = sum p_j v_j; parts of
// a sequence are joined by rescaling with 2^(m_part - m).  m follows the scores
// lazily: it is raised only when a score exceeds it by more than 2^8, so O is
// rescaled a few times per sequence.  p carries a factor of 2^7 (at most 2^15
// as fp16), which keeps weights down to 2^-20 of the largest at fp16's full precision.
//
// What bounds it.  144 bytes per entry for 8192 FLOP (16 heads share K and V):
// HBM, if dequantisation and mma.sync stay behind the copies.  So
//   * the entries of all sequences form one list of 64-entry chunks, of which
//     every CTA (one per SM) takes an equal contiguous share, whatever the
//     lengths; a sequence that spans CTAs leaves partial results that a second
//     kernel joins;
//   * each of eight warps takes every eighth chunk of the share.  It copies its
//     chunks itself, two ahead, into a ring of its own with TMA (codes as
//     128-byte-swizzled boxes of at most a page, scales as one bulk copy per
//     box), so no warp waits for another one;
//   * it dequantises 32 entries at a time in registers straight into mma.sync
//     fragments (E2M1 x E4M3 is exact in fp16) and keeps its own m, l and O,
//     joined once per sequence.  Nothing is written back to shared memory.
// Measured (in a graph; a call from Python adds 1 to 9 us): 8 x 262,144 entries 86 us
// (3.5 TB/s of K, V and scales, 200 TFLOP/s), 1 x 1,048,573 with an fp32 result 75 us,
// 64 sequences of 509 to 32,768 entries 34 us.
// What bounds the long ones is latency: two warps per scheduler (238 registers a thread)
// issue 41 % of the time, and no unit is full (tensor 32 %, ALU 32 %, HBM 38 %).
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace csa2 {

constexpr int DD_WARPS = 8;
constexpr int DD_THREADS = DD_WARPS * 32;
constexpr int DD_CHUNK = 64;                     // entries per chunk
constexpr int DD_UNIT = 32;                      // entries per pass over the registers
constexpr int DD_J = DD_UNIT / 8;                // groups of eight in it
constexpr uint32_t DD_MIN_SHARE = 4;             // places per CTA at least
// A sequence takes a place in the list for each chunk and so many for what it costs
// besides (its Q and the joining of the warps: about 4 us, in which a CTA scores a
// dozen chunks).  A multiple of the warps, so that the next sequence's chunks fall to
// the warps in turn.  64 ragged sequences: 46 us without, 38 with 8 places, 34 with 16;
// 300 short ones 59, 38, 35.
constexpr uint32_t DD_WEIGHT = 16;
static_assert(DD_WEIGHT % DD_WARPS == 0, "whole turns");
constexpr int DD_STAGES = 2;                     // chunks of a warp's ring
constexpr int DD_CODES = DD_CHUNK * kCodeBytes;  // 8 KiB per stage
constexpr int DD_SCALES = DD_CHUNK * kScales;    // 1 KiB
// The tensor core's fp32 sums drop bits at every product, towards zero: a warp's O
// moves to shared memory, where it is added with rounding, after so many chunks.
// fp32 results: four chunks of eight products, 0.6e-6 off at 1M entries instead of 2.0e-6
// (72 us instead of 66; after two chunks 0.4e-6, 79 us).  bf16 results: 64 chunks of four
// products lose 2^-16 at most; without it 3.4e-4 were lost where a CTA has 524,288 entries
// whose V have one sign, a tenth of the result's own step (8 x 262,144 entries 85.4 us
// instead of 84.6).
constexpr uint32_t dd_drain(bool split) { return split ? 4 : 64; }
constexpr int DD_OROW = kD + 4;                  // floats per row of the joining slab (bank spread)
constexpr size_t DD_OFF_CODES = 0;               // [warps][stages]
constexpr size_t DD_OFF_SCALES = DD_OFF_CODES + (size_t)DD_WARPS * DD_STAGES * DD_CODES;
constexpr size_t DD_OFF_SLAB = DD_OFF_SCALES + (size_t)DD_WARPS * DD_STAGES * DD_SCALES;  // [warps][16][DD_OROW] floats
constexpr size_t DD_OFF_M = DD_OFF_SLAB + (size_t)DD_WARPS * kH * DD_OROW * 4;            // [warps][16]
constexpr size_t DD_OFF_L = DD_OFF_M + DD_WARPS * kH * 4;                                 // [warps][16]
constexpr size_t DD_OFF_BAR = DD_OFF_L + DD_WARPS * kH * 4;                               // [warps][stages]
constexpr size_t DD_OFF_MISC = DD_OFF_BAR + DD_WARPS * DD_STAGES * 8;
constexpr size_t DD_SMEM = DD_OFF_MISC + 16;  // start sequence, its first chunk
static_assert(DD_OFF_SCALES % 16 == 0 && DD_OFF_SLAB % 16 == 0 && DD_OFF_BAR % 8 == 0, "dense decode layout");
static_assert(DD_SMEM <= 227 * 1024, "dense decode shared memory");

struct DecodeArgs {
    DenseArgs a;
    float* part_o;  // [2 * ctas][16][128], times 2^(kPBias - m)
    float* part_m;  // [2 * ctas][16] maxima (log2 domain)
    float* part_l;  // [2 * ctas][16] sums
    int4* cut;      // [ctas]: (sequence, its first place, the end of its chunks, first place of this CTA) if it begins inside one
};

// ---- which chunks ---------------------------------------------------------------
// Sequence b's length, 0 if it is out of range.
__device__ __forceinline__ int dense_len(const DenseArgs& a, int b) {
    const int n = __ldg(a.seq_lens + b);
    return n < 0 || n > a.max_len ? 0 : n;
}

__device__ __forceinline__ uint32_t dd_chunks(int n) { return (uint32_t)(n + DD_CHUNK - 1) / DD_CHUNK; }
__device__ __forceinline__ uint32_t dd_places(int n) { return n > 0 ? dd_chunks(n) + DD_WEIGHT : 0u; }
// Offset of 16-byte piece c (0..7) of an entry's row in the swizzled codes
__device__ __forceinline__ uint32_t dd_piece(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

template <bool SPLIT>
__global__ void __launch_bounds__(DD_THREADS, 1)
    dense_decode_kernel(const __grid_constant__ CUtensorMap map, const DecodeArgs d) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const DenseArgs& a = d.a;
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + DD_OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + DD_OFF_BAR) + warp * DD_STAGES;
    if (smem_u32(smem) & 1023u) {  // uniform over the grid
        pdl_wait();
        if (tid == 0) {
            d.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);  // nothing to join
            dev_error(a.err, CSA2_DEV_ALIGN);
        }
        return;
    }
    if (lane == 0) {
        for (int s = 0; s < DD_STAGES; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share: places [lo, hi) of the list -----------------------------
    const int per_thread = (a.B + DD_THREADS - 1) / DD_THREADS;
    const int b0 = min(a.B, tid * per_thread), b1 = min(a.B, b0 + per_thread);
    uint32_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        mine += dd_places(dense_len(a, b));
        if (blockIdx.x == 0) {
            const int n = __ldg(a.seq_lens + b);
            if (n < 0 || n > a.max_len) dev_error(a.err, CSA2_DEV_LEN);
        }
    }
    uint32_t total;
    const uint32_t before = block_excl_scan(mine, reinterpret_cast<uint32_t*>(smem + DD_OFF_SLAB), &total);
    const uint32_t per = max((total + gridDim.x - 1) / gridDim.x, DD_MIN_SHARE);
    const uint32_t lo = min(total, per * blockIdx.x), hi = min(total, lo + per);
    if (lo >= before && lo < before + mine) {
        uint32_t t = before;
        for (int b = b0; b < b1; ++b) {
            const uint32_t n = dd_places(dense_len(a, b));
            if (lo < t + n) {
                misc[0] = (uint32_t)b;
                misc[1] = t;
                break;
            }
            t += n;
        }
    }
    __syncthreads();

    if (lo < hi) {
        // ---- copies: warp w owns chunks lo + w, lo + w + 8, ... and a ring of two -------
        // Nobody else reads the ring: a stage is free when the warp itself has read it.
        const int sh = a.page_shift, box_shift = min(sh, kDenseBoxShift), box = 1 << box_shift, n_box = DD_CHUNK >> box_shift;
        uint8_t* const my_codes = smem + DD_OFF_CODES + (size_t)warp * DD_STAGES * DD_CODES;
        uint8_t* const my_scales = smem + DD_OFF_SCALES + (size_t)warp * DD_STAGES * DD_SCALES;
        int b = (int)misc[0], n = dense_len(a, b);  // the sequence in work: its chunks [t0, te), its places up to t1
        uint32_t t0 = misc[1], te = t0 + dd_chunks(n), t1 = te + DD_WEIGHT;
        int pb = b, pn = n, pos_next = -1;          // the same for the next copy; its box's position (-1: none) ...
        uint32_t p0 = t0, pe = te, c_next = lo + (uint32_t)warp, issued = 0;
        int32_t pg_next = -1;                       // ... and page (not checked yet)
        auto next_seq = [&](int& x) {  // the next sequence that has entries (there is one), its length
            int len;
            do len = dense_len(a, ++x);
            while (len == 0 && x + 1 < a.B);
            return len;
        };
        auto skip = [](uint32_t& c, uint32_t s1) {  // the warp's first place from s1 on
            if (c < s1) c += (s1 - c + DD_WARPS - 1) / DD_WARPS * DD_WARPS;
        };
        auto seek = [&]() {
            while (c_next < hi && c_next >= pe) {  // the next sequence that has chunks
                skip(c_next, pe + DD_WEIGHT);
                if (c_next >= hi) return;
                p0 = pe + DD_WEIGHT;
                pn = next_seq(pb);
                pe = p0 + dd_chunks(pn);
            }
            if (c_next >= hi) return;
            pos_next = (int)(c_next - p0) * DD_CHUNK + lane * box;
            if (lane >= n_box || pos_next >= pn) pos_next = -1;
            else pg_next = __ldg(a.cache.page_table + (int64_t)pb * a.cache.max_pages_per_seq + (pos_next >> sh));
        };
        // the chunk found by seek() into a stage; returns one bit per box that is there
        auto issue = [&](int st) -> uint32_t {
            const bool ok = pos_next >= 0 && pg_next >= 0 && pg_next < a.cache.n_phys_pages;
            if (pos_next >= 0 && !ok) dev_error(a.err, CSA2_DEV_PAGE);
            const uint32_t boxes = __ballot_sync(0xffffffffu, ok);
            if (lane == 0)
                mbar_arrive_expect_tx(&full[st], (uint32_t)__popc(boxes) * (uint32_t)box * (kCodeBytes + kScales));
            __syncwarp();
            if (ok) {
                const int slot = (pg_next << sh) | (pos_next & ((1 << sh) - 1));
                tma_load_2d(my_codes + (size_t)st * DD_CODES + (size_t)lane * box * kCodeBytes, &map, 0, slot, &full[st]);
                bulk_load(my_scales + (size_t)st * DD_SCALES + (size_t)lane * box * kScales,
                          a.cache.scales + (int64_t)slot * kScales, (uint32_t)box * kScales, &full[st]);
            }
            ++issued;
            c_next += DD_WARPS;
            seek();
            return boxes;
        };
        const uint32_t all_boxes = n_box == 32 ? ~0u : (1u << n_box) - 1u;
        uint32_t boxes0 = 0, boxes1 = 0;  // of the chunk in stage 0 and 1
        seek();
        if (c_next < hi) boxes0 = issue(0);
        if (c_next < hi) boxes1 = issue(1);

        const int g = lane >> 2, t4 = lane & 3;
        // Fragment column g (and columns 2 t, 2 t + 1) of an 8-entry group is entry
        // perm(g): its order keeps the swizzled reads of K (16 bytes, lanes g, t)
        // and V (8 bytes, the columns' entries) free of bank conflicts.
        const int kg = ((g >> 1) ^ (((g >> 1) & 1) << 2)) ^ ((g & 1) << 2);
        const int va = t4 ^ ((t4 & 1) << 2), vb = va ^ 4;
        const uint32_t off_k = dd_piece(kg, t4), off_ks = (uint32_t)(kg * kScales + 2 * t4);
        const uint32_t off_va = dd_piece(va, 4 + (g >> 1)) + 8 * (g & 1), off_vb = dd_piece(vb, 4 + (g >> 1)) + 8 * (g & 1);
        const uint32_t off_vs = (uint32_t)(va * kScales + 8 + g);
        float* slab = reinterpret_cast<float*>(smem + DD_OFF_SLAB);
        float* wm = reinterpret_cast<float*>(smem + DD_OFF_M);
        float* wl = reinterpret_cast<float*>(smem + DD_OFF_L);
        if (tid == 0) d.cut[blockIdx.x] = lo > t0 && lo < te ? make_int4(b, (int)t0, (int)te, (int)lo) : make_int4(-1, 0, 0, 0);
        uint32_t t = lo, c = lo + (uint32_t)warp, done = 0;  // c: this warp's chunk, its number `done`
        while (t < hi) {
            if (t >= te) {  // the next sequence that has chunks
                t = t1;
                if (t >= hi) break;
                skip(c, t1);
                n = next_seq(b);
                t0 = t1;
                te = t0 + dd_chunks(n);
                t1 = te + DD_WEIGHT;
            }
            const uint32_t seg0 = t, seg1 = min(hi, te);
            t = seg1;
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

            // this warp's rows of the slab: heads g and g + 8; columns 2 t and 2 t + 1 of tile i
            // are dims 32 t + i and 32 t + 16 + i
            float* my = slab + ((size_t)warp * kH + g) * DD_OROW + 32 * t4;
            // O over f0 and f1, plus what the slab holds (times s0, s1) if `add`
            auto to_slab = [&](float f0, float f1, bool add, float s0, float s1) {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float4* at = reinterpret_cast<float4*>(my + (e >> 1) * 8 * DD_OROW + (e & 1) * 16 + i);
                        const float f = e < 2 ? f0 : f1, sc = e < 2 ? s0 : s1;
                        float4 v = make_float4(O[i][e] * f, O[i + 1][e] * f, O[i + 2][e] * f, O[i + 3][e] * f);
                        if (add) {
                            const float4 u = *at;
                            v = make_float4(fmaf(u.x, sc, v.x), fmaf(u.y, sc, v.y), fmaf(u.z, sc, v.z), fmaf(u.w, sc, v.w));
                        }
                        *at = v;
                    }
            };
            auto ratio = [](float from, float to) { return from == -INFINITY ? 0.f : ex2(from - to); };
            // O moves to the slab; wm holds the maxima that the slab's sums are over
            bool drained = false;
            auto move_out = [&]() {
                to_slab(1.f, 1.f, drained, drained ? ratio(wm[warp * kH + g], m0) : 0.f, drained ? ratio(wm[warp * kH + g + 8], m1) : 0.f);
                __syncwarp();
                if (t4 == 0) wm[warp * kH + g] = m0, wm[warp * kH + g + 8] = m1;
                __syncwarp();
                drained = true;
#pragma unroll
                for (int i = 0; i < 16; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.f;
            };
            uint32_t held = 0;  // chunks in O (fp32 results)

            for (;;) {  // runs of chunks: an fp32 result moves O out inside them, a bf16 one between them
                const uint32_t stop = SPLIT ? seg1 : min(seg1, c + DD_WARPS * dd_drain(SPLIT));
                for (; c < stop; c += DD_WARPS, ++done) {
                    if (SPLIT && held++ == dd_drain(SPLIT)) {
                        held = 1;
                        move_out();
                    }
                    const int st = (int)(done & 1u);
                    if (!mbar_wait(&full[st], (done >> 1) & 1u, a.wait_limit)) {
                        // give up: report, then wait, again with a limit, for the warp's own copies (one or two)
                        if (lane == 0) dev_error(a.err, CSA2_DEV_TIMEOUT);
                        mbar_wait(&full[st], (done >> 1) & 1u, kDenseWaitLimit);
                        if (issued > done + 1) mbar_wait(&full[st ^ 1], ((done + 1) >> 1) & 1u, kDenseWaitLimit);
                        c = c_next = hi;
                        break;
                    }
                    const uint8_t* codes = my_codes + (size_t)st * DD_CODES;
                    uint8_t* scales = my_scales + (size_t)st * DD_SCALES;
                    const uint32_t boxes = st ? boxes1 : boxes0;
                    const int left = n - (int)(c - t0) * DD_CHUNK;  // entries from the chunk's first on
                    // Entries that are not there (behind the last one, of a missing page) get scale
                    // 0, so K and V are 0; their scores are hidden below.
                    const bool partial = boxes != all_boxes || left < DD_CHUNK;
                    auto gone = [&](int e) { return e >= left || !((boxes >> (e >> box_shift)) & 1u); };
                    if (partial) {
#pragma unroll
                        for (int e = lane; e < DD_CHUNK; e += 32)
                            if (gone(e)) *reinterpret_cast<uint4*>(scales + e * kScales) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();  // the next copy into the stage comes after these writes
                        __syncwarp();
                    }
#pragma unroll
                    for (int u0 = 0; u0 < DD_CHUNK; u0 += DD_UNIT, codes += DD_UNIT * kCodeBytes, scales += DD_UNIT * kScales) {
                        // ---- S = Q K^T, four groups of eight entries ---------------------------------
                        float S[DD_J][4];
                        {
                            uint4 kc[DD_J];
                            uint32_t kl[DD_J], kh[DD_J];
#pragma unroll
                            for (int j = 0; j < DD_J; ++j) {
                                kc[j] = *reinterpret_cast<const uint4*>(codes + j * 8 * kCodeBytes + off_k);
                                const uint32_t s2 = e4m3x2_to_h2(*reinterpret_cast<const uint16_t*>(scales + j * 8 * kScales + off_ks));
                                kl[j] = __byte_perm(s2, 0u, 0x1010);
                                kh[j] = __byte_perm(s2, 0u, 0x3232);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t x[DD_J][4];
#pragma unroll
                                for (int j = 0; j < DD_J; ++j) {
                                    const uint32_t w = i == 0 ? kc[j].x : i == 1 ? kc[j].y : i == 2 ? kc[j].z : kc[j].w;
                                    e2m1x8_to_h2x4(w, x[j][0], x[j][1], x[j][2], x[j][3]);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) x[j][e] = hmul2(x[j][e], i < 2 ? kl[j] : kh[j]);
                                }
                                // group by group, so that four products lie between two of one sum
#pragma unroll
                                for (int j = 0; j < DD_J; ++j) {
                                    if (i == 0) mma16816_zero(S[j], qa[0], x[j][0], x[j][1]);
                                    else mma16816(S[j], qa[2 * i], x[j][0], x[j][1]);
                                }
#pragma unroll
                                for (int j = 0; j < DD_J; ++j) mma16816(S[j], qa[2 * i + 1], x[j][2], x[j][3]);
                            }
                        }
                        uint2 vc[DD_J][2];
                        uint32_t vs[DD_J];  // scales of entries va and vb
#pragma unroll
                        for (int j = 0; j < DD_J; ++j) {
                            vc[j][0] = *reinterpret_cast<const uint2*>(codes + j * 8 * kCodeBytes + off_va);
                            vc[j][1] = *reinterpret_cast<const uint2*>(codes + j * 8 * kCodeBytes + off_vb);
                            vs[j] = (uint32_t)scales[j * 8 * kScales + off_vs] |
                                    ((uint32_t)scales[j * 8 * kScales + (off_vs ^ (4 * kScales))] << 8);
                        }
                        if (u0 + DD_UNIT == DD_CHUNK) {  // the stage is in registers: the chunk after next goes there
                            __syncwarp();
                            if (c_next < hi) {
                                const uint32_t x = issue(st);
                                if (st) boxes1 = x;
                                else boxes0 = x;
                            }
                        }
                        // ---- weights: log2 domain, minus the maximum plus kPBias ------------------------
#pragma unroll
                        for (int j = 0; j < DD_J; ++j) {
                            S[j][0] = fmaf(S[j][0], c0, bias0);
                            S[j][1] = fmaf(S[j][1], c0, bias0);
                            S[j][2] = fmaf(S[j][2], c1, bias1);
                            S[j][3] = fmaf(S[j][3], c1, bias1);
                        }
                        float mx0 = fmaxf(S[0][0], S[0][1]), mx1 = fmaxf(S[0][2], S[0][3]);
#pragma unroll
                        for (int j = 1; j < DD_J; ++j) {
                            mx0 = fmaxf(fmaxf(mx0, S[j][0]), S[j][1]);
                            mx1 = fmaxf(fmaxf(mx1, S[j][2]), S[j][3]);
                        }
                        if (__any_sync(0xffffffffu, partial || fmaxf(mx0, mx1) > kPMax || fminf(m0, m1) == -INFINITY)) {
                            mx0 = mx1 = -INFINITY;
#pragma unroll
                            for (int j = 0; j < DD_J; ++j) {
                                if (partial && gone(u0 + 8 * j + va)) S[j][0] = S[j][2] = -INFINITY;
                                if (partial && gone(u0 + 8 * j + vb)) S[j][1] = S[j][3] = -INFINITY;
                                mx0 = fmaxf(mx0, fmaxf(S[j][0], S[j][1]));
                                mx1 = fmaxf(mx1, fmaxf(S[j][2], S[j][3]));
                            }
                            mx0 = quad_max(mx0) - bias0;  // the scores' maxima
                            mx1 = quad_max(mx1) - bias1;
                            const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
                            const float nb0 = n0 == -INFINITY ? kPBias : kPBias - n0, nb1 = n1 == -INFINITY ? kPBias : kPBias - n1;
                            const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
#pragma unroll
                            for (int j = 0; j < DD_J; ++j) {
                                S[j][0] += nb0 - bias0;
                                S[j][1] += nb0 - bias0;
                                S[j][2] += nb1 - bias1;
                                S[j][3] += nb1 - bias1;
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
                        uint32_t pa[DD_J / 2][4], pl[DD_J / 2][4];
#pragma unroll
                        for (int j = 0; j < DD_J; ++j) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) S[j][e] = ex2(S[j][e]);
                            l0 += S[j][0] + S[j][1];
                            l1 += S[j][2] + S[j][3];
                            uint32_t* p = &pa[j >> 1][2 * (j & 1)];
                            p[0] = f2_to_h2(S[j][0], S[j][1]);
                            p[1] = f2_to_h2(S[j][2], S[j][3]);
                            if (SPLIT) {  // what the first fp16 term leaves
                                pl[j >> 1][2 * (j & 1)] = rest_h2(S[j][0], S[j][1], p[0]);
                                pl[j >> 1][2 * (j & 1) + 1] = rest_h2(S[j][2], S[j][3], p[1]);
                            }
                        }
                        // ---- O += P V: tile 8 w + i of eight columns g is dims 16 g + 8 w + i ------------
#pragma unroll
                        for (int u = 0; u < DD_J / 2; ++u) {  // sixteen entries
                            const uint32_t sc0 = e4m3x2_to_h2(vs[2 * u]), sc1 = e4m3x2_to_h2(vs[2 * u + 1]);
#pragma unroll
                            for (int w = 0; w < 2; ++w) {
                                // nibble pairs (entry va, entry vb) of one dim in one byte: even dims, then odd dims
                                uint32_t x[2][8];
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const uint2 a2 = vc[2 * u + j][0], b2 = vc[2 * u + j][1];
                                    const uint32_t p = w ? a2.y : a2.x, q = w ? b2.y : b2.x;
                                    const uint32_t ev = (p & 0x0f0f0f0fu) | ((q << 4) & 0xf0f0f0f0u);
                                    const uint32_t od = ((p >> 4) & 0x0f0f0f0fu) | (q & 0xf0f0f0f0u);
                                    e2m1x8_to_h2x4(ev, x[j][0], x[j][2], x[j][4], x[j][6]);
                                    e2m1x8_to_h2x4(od, x[j][1], x[j][3], x[j][5], x[j][7]);
                                }
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    x[0][i] = hmul2(x[0][i], sc0);
                                    x[1][i] = hmul2(x[1][i], sc1);
                                    mma16816(O[8 * w + i], pa[u], x[0][i], x[1][i]);
                                }
                                if (SPLIT)
#pragma unroll
                                    for (int i = 0; i < 8; ++i)  // V / kLoScale, exact
                                        mma16816(O[8 * w + i], pl[u], hmul2(x[0][i], 0x0c000c00u), hmul2(x[1][i], 0x0c000c00u));
                            }
                        }
                    }
                }
                if (SPLIT || c >= seg1) break;
                move_out();
            }

            // ---- join the warps' results of the segment ------------------------------
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            const float s0 = drained ? wm[warp * kH + g] : -INFINITY, s1 = drained ? wm[warp * kH + g + 8] : -INFINITY;
            __syncwarp();
            if (t4 == 0) {
                wm[warp * kH + g] = m0;
                wm[warp * kH + g + 8] = m1;
                wl[warp * kH + g] = l0;
                wl[warp * kH + g + 8] = l1;
            }
            __syncthreads();
            float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
            for (int w = 0; w < DD_WARPS; ++w) {
                M0 = fmaxf(M0, wm[w * kH + g]);
                M1 = fmaxf(M1, wm[w * kH + g + 8]);
            }
            to_slab(ratio(m0, M0), ratio(m1, M1), drained, ratio(s0, M0), ratio(s1, M1));
            __syncthreads();
            if (tid < kH * 16) {
                const int h = tid >> 4, d8 = (tid & 15) * 8;  // 16 heads x 16 threads of 8 dims
                float M = -INFINITY, l = 0.f, o[8];
#pragma unroll
                for (int w = 0; w < DD_WARPS; ++w) M = fmaxf(M, wm[w * kH + h]);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll
                for (int w = 0; w < DD_WARPS; ++w) {
                    const float mw = wm[w * kH + h];
                    l += mw == -INFINITY ? wl[w * kH + h] : wl[w * kH + h] * ex2(mw - M);  // (0, or the NaN of scores that all are)
                }
#pragma unroll
                for (int w = 0; w < DD_WARPS; ++w) {
                    const float* p = slab + ((size_t)w * kH + h) * DD_OROW + d8;
                    const float4 v0 = *reinterpret_cast<const float4*>(p), v1 = *reinterpret_cast<const float4*>(p + 4);
                    o[0] += v0.x, o[1] += v0.y, o[2] += v0.z, o[3] += v0.w;
                    o[4] += v1.x, o[5] += v1.y, o[6] += v1.z, o[7] += v1.w;
                }
                if (seg0 == t0 && seg1 == te) {  // the whole sequence
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
            __syncthreads();  // the slab is free for the next segment
        }
    } else if (tid == 0) {
        d.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    // sequences without entries
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
        if (tid < kH * 16 && dense_len(a, b) == 0) {
            const float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            dense_store(a, (int64_t)b * kH + (tid >> 4), (tid & 15) * 8, o, -INFINITY, 0.f);
        }
}

// Joins the partial results of every sequence that spans CTAs: block (c, y) the
// heads 4 y .. 4 y + 3 of the sequence that CTA c continues, if CTA c - 1 began
// it.  Four warps per head share the parts; sums in a fixed order.
constexpr int DJ_THREADS = 512;
__global__ void __launch_bounds__(DJ_THREADS) dense_decode_join_kernel(const DecodeArgs d) {
    __shared__ float4 s_o[16][32];
    const DenseArgs& a = d.a;
    const int c = blockIdx.x + 1, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_trigger();
    const int4 cut = d.cut[c];
    if (cut.x < 0) return;
    const int per = cut.w / c;  // CTA c begins at place c * per
    if (cut.y < (c - 1) * per) return;  // an earlier CTA's block does it
    const int last = (cut.z - 1) / per, n = last - c + 2;
    const int h = 4 * blockIdx.y + (warp >> 2), w4 = warp & 3;
    auto part = [&](int k) { return (int64_t)(k == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + k)) * kH + h; };
    // lane k holds the factors of parts k, k + 32, ..., so only the rows are read in the loop
    constexpr int SLOTS = (kDenseCtas + 31) / 32;
    float f[SLOTS], pl[SLOTS], M = -INFINITY, l = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        f[s] = lane + 32 * s < n ? d.part_m[part(lane + 32 * s)] : -INFINITY;
        pl[s] = lane + 32 * s < n ? d.part_l[part(lane + 32 * s)] : 0.f;
        M = fmaxf(M, f[s]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        f[s] = f[s] == -INFINITY ? 0.f : ex2(f[s] - M);
        l += pl[s] * f[s];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
#pragma unroll 8
        for (int k = 32 * s + w4; k < min(n, 32 * s + 32); k += 4) {
            const float4 v = *reinterpret_cast<const float4*>(d.part_o + part(k) * kD + 4 * lane);
            const float g = __shfl_sync(0xffffffffu, f[s], k & 31);
            o.x += v.x * g;
            o.y += v.y * g;
            o.z += v.z * g;
            o.w += v.w * g;
        }
    s_o[warp][lane] = o;
    __syncthreads();
    if (w4 == 0 && lane < 16) {
        float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float4 x = s_o[warp + w][2 * lane], y = s_o[warp + w][2 * lane + 1];
            r[0] += x.x, r[1] += x.y, r[2] += x.z, r[3] += x.w;
            r[4] += y.x, r[5] += y.y, r[6] += y.z, r[7] += y.w;
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
    if (!dense_code_map(a.cache, &map)) return cudaErrorInvalidValue;
    DecodeArgs d{};
    d.a = a;
    float* f = reinterpret_cast<float*>(ws);
    d.part_o = f;
    d.part_m = d.part_o + (size_t)2 * kDenseCtas * kH * kD;
    d.part_l = d.part_m + (size_t)2 * kDenseCtas * kH;
    d.cut = reinterpret_cast<int4*>(d.part_l + (size_t)2 * kDenseCtas * kH);
    const int64_t most = (int64_t)a.B * ((a.max_len + DD_CHUNK - 1) / DD_CHUNK + DD_WEIGHT);  // places there can be
    const unsigned ctas = (unsigned)std::min<int64_t>(std::min(n_sm[dev], kDenseCtas), most);
    LaunchCfg c(dim3(ctas), dim3(DD_THREADS), DD_SMEM, stream);
    e = a.out_bf16 ? cudaLaunchKernelEx(&c.cfg, dense_decode_kernel<false>, (const CUtensorMap)map, d)
                   : cudaLaunchKernelEx(&c.cfg, dense_decode_kernel<true>, (const CUtensorMap)map, d);
    if (e != cudaSuccess || ctas == 1) return e;
    LaunchCfg j(dim3(ctas - 1, kH / 4), dim3(DJ_THREADS), 0, stream);
    return cudaLaunchKernelEx(&j.cfg, dense_decode_join_kernel, d);
}

}  // namespace csa2

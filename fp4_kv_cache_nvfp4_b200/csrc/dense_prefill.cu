// Dense prefill attention on the 5th-generation tensor cores (tcgen05): ragged
// chunks of query tokens over every entry of the FP4 main KV that they see.
//
// Mathematics as in decode: one pass over the entries with a running maximum
// and sum per row, the maximum following lazily (see dense_decode.cu).  A row
// is a (token, head) pair: the 16 heads share K and V, so 8 tokens fill the 128
// rows of a product,
//   S[128 x 128 entries] = Q . K^T,   O[128 x 128 dims] += P . V.
//
// A work unit is 16 tokens (two 128-row tiles) over its tiles of 128 entries.
// The tiles of all units form one list, of which every CTA (one per SM) takes an
// equal contiguous share, whatever the lengths and masks; a unit that spans
// CTAs leaves partial results that a second kernel joins.  In a CTA
//   warps 0-3, 4-7  softmax of row tile 0 and 1, one thread per row: maximum,
//                   P = 2^(S c - m) as fp16 back into TMEM over S, the sum;
//                   O's rescaling when m rises (rare); the result's rows
//   4 or 6 more     K and V of the next tiles: FP4 read with plain loads one tile
//                   ahead, dequantised to fp16 (exact) into swizzled shared tiles
//   the last one    issues the products: while one row tile is in its softmax, the
//                   other's products run
// TMEM: S of both row tiles (P over them), O of both: all 512 columns.
//
// What bounds it: latency.  Per (row tile, entry tile) the products take 1024 cycles of
// the tensor core and the 16,384 exponentials 1024 cycles of the special-function units,
// but a pair of row tiles takes 4,170 cycles, not 2,048: the chain S -> softmax -> P ->
// products of a row tile is serial, and two row tiles fill TMEM.  Both units are busy
// 47 % of the time, instructions issue 41 %.  At 128 registers a thread all four kernels
// spill (220 to 290 bytes stored).
// Measured (in a graph): the last 4096 of 32,768 tokens at ratio 2 (16,384 entries) 486
// us, 1060 TFLOP/s of the products that the mask leaves; in a run of seconds the power cap
// lowers the clock from 1965 to 1850 MHz, and a call takes 523 us.  Drafts of 8 x 5
// tokens over 65,536 entries 69 us.
#include <string.h>

#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace csa2 {

constexpr int DP_TOK = 16;                       // tokens per unit (8 per row tile)
constexpr uint32_t DP_WEIGHT = 3;                // places of a unit besides its tiles': ragged prompts 124 us with 1, 103 with 3
constexpr int DP_ROWS = DP_TOK * kH;             // 256
constexpr int DP_KEYS = 128;                     // entries per tile
constexpr uint32_t DP_HALF = 128 * 128;          // 64 channels of an operand tile: [128 rows][128 B], swizzled
constexpr uint32_t DP_TILE = 2 * DP_HALF;        // 32 KiB
constexpr int DP_W_CONV = 8;                     // the first converter warp; the one that issues follows the last
// Converter warps.  Sixteen warps leave a thread 128 registers, as thirteen do.  The
// paired kernel takes an entry tile for one row tile, not for two, and waits for the
// conversion: with four 73.5 us (8 x 5 tokens over 65,536 entries), with six 69.4, with
// seven 69.4; without pairs four 486 us (4096 over 16,384 entries), six 516: they
// issue beside the softmax.  With three (168 registers, no spills) 82 and 513.
constexpr int dp_conv(bool paired) { return paired ? 6 : 4; }
constexpr int dp_threads(bool paired) { return (DP_W_CONV + dp_conv(paired) + 1) * 32; }
constexpr size_t DP_OFF_Q = 0;                            // [2 row tiles]
constexpr size_t DP_OFF_K = DP_OFF_Q + 2 * DP_TILE;       // [2 slots]
constexpr size_t DP_OFF_V = DP_OFF_K + 2 * DP_TILE;       // [2 slots]
constexpr size_t DP_OFF_OK = DP_OFF_V + 2 * DP_TILE;      // [4][16 B]: one bit per entry of a K tile, 0: missing page
constexpr size_t DP_OFF_ML = DP_OFF_OK + 64;              // [128] (m, l) of the second group's rows
constexpr size_t DP_OFF_BAR = DP_OFF_ML + 1024;
constexpr int DP_NBAR = 4 * 2 + 4 * 2 + 1;
constexpr size_t DP_OFF_SCAN = DP_OFF_BAR + DP_NBAR * 8;  // [64] words
constexpr size_t DP_OFF_MISC = DP_OFF_SCAN + 256;         // tmem base, timeout flag, start sequence, unit, its first tile
constexpr size_t DP_SMEM = DP_OFF_MISC + 32 + 1024;       // + slack for the 1 KiB alignment
static_assert(DP_OFF_BAR % 8 == 0 && DP_SMEM <= 227 * 1024, "dense prefill layout");
constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
constexpr uint32_t kIdescPV = kIdescS | (1u << 16);  // B (V) has its dims contiguous

// The tensor core's fp32 sums drop bits at every product, towards zero, so O's bias
// grows with its tiles.  After so many tiles of a row tile, O is added, with rounding,
// to sums in the workspace (they stay in L2), and the products begin anew.
// fp32 results, 9 x 256 tokens over 16,384 entries (in a graph): every two tiles 5.4e-7
// off and 627 us, every four 1.1e-6 and 551 us, every tile 3.4e-7 and 755 us, never 2.7e-5.
// bf16 results: 64 tiles of 8 products lose 2^-15 at most, 1/128 of the result's own
// step; without it 7.2e-4 were lost over 262,144 entries whose V have one sign, a sixth
// of a step.  4096 tokens over 16,384 entries 485 us instead of 479.
constexpr uint32_t dp_drain(bool split) { return split ? 2 : 64; }

struct PrefillDenseArgs {
    DenseArgs a;
    float4* sums;   // [ctas][2 row tiles][32 groups of 4 dims][128 rows]
    float* part_o;  // [2 * ctas][256 rows][128], times 2^(kPBias - m)
    float* part_m;  // [2 * ctas][256]
    float* part_l;  // [2 * ctas][256]
    int4* cut;      // [2 * ctas]: (first row token, tokens, first place, end of the tiles), (first place of this CTA) of the unit it begins inside
};

// ---- which units and tiles ----------------------------------------------------------
// One sequence's queries: tokens [row0, row0 + nq), the first at position p0.
struct SeqQ {
    int row0, nq, len;
    int64_t p0;
    __device__ __forceinline__ int units() const { return (nq + DP_TOK - 1) / DP_TOK; }
};
__device__ __forceinline__ SeqQ seq_q(const DenseArgs& a, int b, bool report) {
    SeqQ s;
    const int lo = __ldg(a.cu_q + b), hi = __ldg(a.cu_q + b + 1);
    const bool range = lo >= 0 && hi >= lo && hi <= a.T;
    s.row0 = lo;
    s.nq = range ? hi - lo : 0;
    s.len = __ldg(a.seq_lens + b);
    s.p0 = a.q_start ? __ldg(a.q_start + b) : 0;
    const bool bad = s.len < 0 || s.len > a.max_len || s.p0 < 0;
    if (report && (!range || bad)) dev_error(a.err, CSA2_DEV_LEN);
    if (bad) {
        s.len = 0;
        s.p0 = 0;
    }
    return s;
}
// Entries that the token `i` of the sequence sees
__device__ __forceinline__ int seen_by(const DenseArgs& a, const SeqQ& s, int i) {
    if (!a.q_start) return s.len;
    const int64_t v = (s.p0 + i + 1) >> (a.ratio - 1);
    return v < s.len ? (int)v : s.len;
}
// Entries that unit k's last token sees, and the tiles they take, one at least (it writes the rows)
__device__ __forceinline__ int unit_seen(const DenseArgs& a, const SeqQ& s, int k) {
    return seen_by(a, s, min((k + 1) * DP_TOK, s.nq) - 1);
}
__device__ __forceinline__ uint32_t tiles_of(int seen) { return max(1u, (uint32_t)(seen + DP_KEYS - 1) / DP_KEYS); }
__device__ __forceinline__ uint32_t unit_tiles(const DenseArgs& a, const SeqQ& s, int k) { return tiles_of(unit_seen(a, s, k)); }
// Places in the list of the units before k: a unit takes one for each tile and
// DP_WEIGHT for what it costs besides (its Q, its rows: as long as a tile or two,
// which counts where the units are short).  With A = p0 + 16 + 127 r and D = 128 r, a
// full unit i has min(C, floor((A + 16 i) / D)) tiles, C = ceil(len / 128): a
// staircase, whose sum is a difference of G(x) = sum_{j < x} floor(j / (8 r)).
__device__ __forceinline__ uint64_t places_before(const DenseArgs& a, const SeqQ& s, int k) {
    if (k <= 0) return 0;
    const int last = s.units() - 1;
    const uint64_t C = max(1u, (uint32_t)(s.len + DP_KEYS - 1) / DP_KEYS);
    const int m = min(k, last);  // full units
    uint64_t n;
    if (!a.q_start) {
        n = (uint64_t)m * C;
    } else {
        const int r = a.ratio, sh = 3 + (r - 1);  // 8 r = 2^sh
        const int64_t A = s.p0 + DP_TOK + 127 * r, x = A >> 4;
        int64_t ic = ((int64_t)(C << (sh + 4)) - A + DP_TOK - 1) >> 4;  // the first unit with C
        ic = ic < 0 ? 0 : ic > m ? m : ic;
        auto G = [&](int64_t v) {
            const int64_t q = v >> sh;
            return ((q * (q - 1) / 2) << sh) + q * (v - (q << sh));
        };
        n = (uint64_t)(G(x + ic) - G(x)) + (uint64_t)(m - ic) * C;
    }
    return (k > last ? n + unit_tiles(a, s, last) : n) + (uint64_t)k * DP_WEIGHT;
}

// Walks the units of a CTA's share in order.
struct Walk {
    int b, k, nk;
    SeqQ s;
    int seen;         // entries that some token of the unit sees
    uint32_t t0, te;  // the unit's tiles in the list; its other places follow
    __device__ __forceinline__ void start(const DenseArgs& a, const uint32_t* at) {
        b = (int)at[0];
        k = (int)at[1];
        t0 = at[2];
        s = seq_q(a, b, false);
        nk = s.units();
        seen = unit_seen(a, s, k);
        te = t0 + tiles_of(seen);
    }
    __device__ __forceinline__ void next(const DenseArgs& a) {
        t0 = te + DP_WEIGHT;
        if (++k >= nk) {
            k = 0;
            do {
                s = seq_q(a, ++b, false);
                nk = s.units();
            } while (nk == 0 && b + 1 < a.B);
        }
        seen = unit_seen(a, s, k);
        te = t0 + tiles_of(seen);
    }
    // The first tile at or behind place t, and the end of the CTA's tiles of its unit.
    // False: there is none before hi.
    __device__ __forceinline__ bool tiles(const DenseArgs& a, uint32_t& t, uint32_t hi, uint32_t& end) {
        if (t < hi && t >= te) {
            t = te + DP_WEIGHT;
            if (t < hi) next(a);
        }
        end = min(hi, te);
        return t < hi;
    }
    __device__ __forceinline__ int tokens() const { return min(DP_TOK, s.nq - k * DP_TOK); }
    // A unit of one row tile: the two groups of softmax warps take its entry tiles in
    // turn, each with its own O, and join them at the end.
    template <bool PAIRED>
    __device__ __forceinline__ bool split(uint32_t t, uint32_t end) const {
        return PAIRED && tokens() <= DP_TOK / 2 && end - t >= 2;
    }
};

// ---- tensor-core helpers --------------------------------------------------------------
// Descriptors as two words, so that a step along K is one addition to the low
// one (see umma_desc_sw128, umma_desc_sw128_mn): the thread that issues the
// products has little time for address arithmetic.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (uint32_t)umma_desc_sw128(saddr); }
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t saddr) { return (uint32_t)umma_desc_sw128_mn(saddr, DP_HALF); }
// D[128 x 128] (+)= A . B with fp16 operands, A in shared memory
__device__ __forceinline__ void dp_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kIdescS), "r"(kDescHi), "r"(acc)
        : "memory");
}
// the same with A in TMEM (rows = lanes, two fp16 per column) and B transposed
__device__ __forceinline__ void dp_mma_ts(uint32_t d, uint32_t ta, uint32_t b, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 db, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(ta), "r"(b), "r"(kIdescPV), "r"(kDescHi), "r"(acc)
        : "memory");
}
// the same, D = D * 2^-12 + A . B (kLoScale)
__device__ __forceinline__ void dp_mma_ts_lo_done(uint32_t d, uint32_t ta, uint32_t b) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.eq.b32 p, 0, 0;\n\tmov.b64 db, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p, 12;\n\t}" ::"r"(d),
        "r"(ta), "r"(b), "r"(kIdescPV), "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// 32 consecutive columns of this thread's lane
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t (&v)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
          "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
          "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
          "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
          "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
        "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// SPLIT: P as two fp16 terms (fp32 results).  PAIRED: units of one row tile use
// both groups of softmax warps.
template <bool SPLIT, bool PAIRED>
__global__ void __launch_bounds__(dp_threads(PAIRED), 1) dense_prefill_kernel(const PrefillDenseArgs d) {
    constexpr int NCONV = dp_conv(PAIRED), W_MMA = DP_W_CONV + NCONV;
    constexpr int STEP = NCONV * 8, ENT = (DP_KEYS + STEP - 1) / STEP;  // a converter thread has at most ENT entries, STEP apart
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const DenseArgs& a = d.a;
    uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + DP_OFF_BAR);  // [2] K tile written (converter warps)
    uint64_t* kempty = kfull + 2;                                      // [2] read by the products (commit)
    uint64_t* vfull = kempty + 2;
    uint64_t* vempty = vfull + 2;
    uint64_t* qfull = vempty + 2;   // [2] a row tile's Q written (4 softmax warps)
    uint64_t* sfull = qfull + 2;    // [2] S complete (commit)
    uint64_t* pfull = sfull + 2;    // [2] P written, O rescaled (4 softmax warps)
    uint64_t* ofull = pfull + 2;    // [2] O of a unit complete (commit)
    uint64_t* mma_done = ofull + 2;
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + DP_OFF_MISC);
    volatile uint32_t* s_timeout = misc + 1;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kfull[i], NCONV);
            mbar_init(&kempty[i], 1);
            mbar_init(&vfull[i], NCONV);
            mbar_init(&vempty[i], 1);
            mbar_init(&qfull[i], 4);
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&ofull[i], 1);
        }
        mbar_init(mma_done, 1);
        *s_timeout = 0;
        fence_mbar_init();
    }
    if (wid == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(misc)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share: places [lo, hi) of the list -----------------------------
    const int per_thread = (a.B + (int)blockDim.x - 1) / (int)blockDim.x;
    const int b0 = min(a.B, tid * per_thread), b1 = min(a.B, b0 + per_thread);
    uint64_t sum = 0;
    bool ascending = true;
    for (int b = b0; b < b1; ++b) {
        const SeqQ s = seq_q(a, b, blockIdx.x == 0);
        sum += places_before(a, s, s.units());
        ascending &= __ldg(a.cu_q + b) <= __ldg(a.cu_q + b + 1);
    }
    const uint32_t mine = (uint32_t)sum;
    uint32_t total;
    const uint32_t before = block_excl_scan(mine, reinterpret_cast<uint32_t*>(smem + DP_OFF_SCAN), &total);
    // The host's bound on the places holds while no ranges overlap, which only a range
    // that is not ascending makes possible.  Then the places are counted again, in units
    // of 2^16 (rounded down: below 2^15 of them the sum above has not wrapped), and a
    // call whose places do not fit does nothing.
    if (__syncthreads_or(!ascending)) {
        uint32_t coarse;
        block_excl_scan((uint32_t)min(sum >> 16, (uint64_t)1 << 16), reinterpret_cast<uint32_t*>(smem + DP_OFF_SCAN), &coarse);
        if (coarse >= 1u << 15 || total > (uint32_t)INT32_MAX) {
            total = 0;
            if (tid == 0) dev_error(a.err, CSA2_DEV_LEN);
        }
    }
    const uint32_t per = (total + gridDim.x - 1) / gridDim.x;
    const uint32_t lo = min(total, per * blockIdx.x), hi = min(total, lo + per);
    if (lo < hi && lo >= before && lo < before + mine) {
        uint32_t t = before;
        for (int b = b0; b < b1; ++b) {
            const SeqQ s = seq_q(a, b, false);
            const uint32_t n = (uint32_t)places_before(a, s, s.units());
            if (lo < t + n) {
                int k0 = 0, k1 = s.units();  // the last unit whose first tile is not behind lo
                while (k1 - k0 > 1) {
                    const int k = (k0 + k1) / 2;
                    if (places_before(a, s, k) <= lo - t) k0 = k;
                    else k1 = k;
                }
                misc[2] = (uint32_t)b;
                misc[3] = (uint32_t)k0;
                misc[4] = t + (uint32_t)places_before(a, s, k0);
                break;
            }
            t += n;
        }
    }
    __syncthreads();
    // bounded; a thread that gave up once does not wait any more
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, a.wait_limit)) {
            dead = true;
            *s_timeout = 1;
        }
    };

    if (lo < hi && wid == W_MMA) {
        // ================= the products: every lane keeps the books, one issues =================
        const bool leader = elect_one();
        Walk w;
        w.start(a, misc + 2);
        uint32_t ks = 0, kph = 0, vs = 0, vph = 0, qph = 0, qph1 = 0, pph0 = 0, pph1 = 0;  // slots and phases
        const uint32_t qlo = desc_lo(smem_u32(smem + DP_OFF_Q)), klo = desc_lo(smem_u32(smem + DP_OFF_K)),
                       vlo = desc_lo_mn(smem_u32(smem + DP_OFF_V));
        auto mma_s = [&](int i, int qi) {  // S i: row tile qi over the K tile in slot ks
            if (leader) {
                const uint32_t q = qlo + (uint32_t)qi * (DP_TILE >> 4), k = klo + ks * (DP_TILE >> 4);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint32_t o = (uint32_t)(x >> 2) * (DP_HALF >> 4) + 2u * (x & 3);
                    dp_mma_ss(tmem + 128u * i, q + o, k + o, x > 0);
                }
                umma_commit(&sfull[i]);
            }
            __syncwarp();
        };
        auto mma_pv = [&](int i, bool first) {  // O of row tile i += P . V tile in slot vs
            if (leader) {
                const uint32_t v = vlo + vs * (DP_TILE >> 4), p = tmem + 128u * i, o = tmem + 256u + 128u * i;
                if (SPLIT) {  // the low terms on kLoScale * O, then O = that / kLoScale + the high terms
#pragma unroll
                    for (int x = 0; x < 8; ++x) dp_mma_ts(o, p + 32u * (x >> 1) + 16u + 8u * (x & 1), v + 128u * x, x > 0 || !first);
                    dp_mma_ts_lo_done(o, p, v);
#pragma unroll
                    for (int x = 1; x < 8; ++x) dp_mma_ts(o, p + 32u * (x >> 1) + 8u * (x & 1), v + 128u * x, 1);
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x)  // P of 16 entries: 8 columns
                        dp_mma_ts(o, p + 32u * (x >> 1) + 8u * (x & 1), v + 128u * x, x > 0 || !first);
                }
            }
            __syncwarp();
        };
        // the k-th tile of a row tile (or group) begins O
        auto fresh = [](uint32_t k) { return k % dp_drain(SPLIT) == 0; };
        auto commit = [&](uint64_t* bar) {
            if (leader) umma_commit(bar);
            __syncwarp();
        };
        auto next_k = [&]() {
            commit(&kempty[ks]);
            ks ^= 1u;
            kph ^= ks == 0;
        };
        for (uint32_t t = lo, end; w.tiles(a, t, hi, end);) {
            const bool two = w.tokens() > DP_TOK / 2;
            wait(&qfull[0], qph);
            qph ^= 1u;
            if (w.split<PAIRED>(t, end)) {
                const uint32_t first = t;
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    wait(&kfull[ks], kph);
                    tc_fence_after();
                    mma_s(i, 0);
                    next_k();
                }
#pragma unroll 1
                for (; t < end; ++t) {
                    const int i = (int)(t - first) & 1;
                    wait(&vfull[vs], vph);
                    wait(&pfull[i], i ? pph1 : pph0);
                    if (i) pph1 ^= 1u;
                    else pph0 ^= 1u;
                    tc_fence_after();
                    mma_pv(i, fresh((t - first) >> 1));
                    commit(&vempty[vs]);
                    vs ^= 1u;
                    vph ^= vs == 0;
                    if (t + 2 < end) {
                        wait(&kfull[ks], kph);
                        tc_fence_after();
                        mma_s(i, 0);
                        next_k();
                    } else {
                        commit(&ofull[i]);
                    }
                }
                continue;
            }
            if (two) {
                wait(&qfull[1], qph1);
                qph1 ^= 1u;
            }
            wait(&kfull[ks], kph);
            tc_fence_after();
            mma_s(0, 0);
            if (two) mma_s(1, 1);
            next_k();
            for (const uint32_t first = t; t < end; ++t) {
                const bool more = t + 1 < end;
                wait(&vfull[vs], vph);
                wait(&pfull[0], pph0);
                pph0 ^= 1u;
                tc_fence_after();
                mma_pv(0, fresh(t - first));
                if (more) {
                    wait(&kfull[ks], kph);
                    tc_fence_after();
                    mma_s(0, 0);
                } else {
                    commit(&ofull[0]);
                }
                if (two) {
                    wait(&pfull[1], pph1);
                    pph1 ^= 1u;
                    tc_fence_after();
                    mma_pv(1, fresh(t - first));
                }
                commit(&vempty[vs]);
                vs ^= 1u;
                vph ^= vs == 0;
                if (more) {
                    if (two) mma_s(1, 1);
                    next_k();
                } else if (two) {
                    commit(&ofull[1]);
                }
            }
        }
        commit(mma_done);
        // whatever was given up above: the products in flight end before TMEM is freed
        if (!mbar_wait(mma_done, 0u, kDenseWaitLimit)) *s_timeout = 1;
    } else if (lo < hi && wid >= DP_W_CONV) {
        // ================= converters: FP4 rows -> fp16 operand tiles =================
        // Thread ct owns quarter qt (32 channels of K and of V) of entries e0 + STEP i.
        const int ct = tid - DP_W_CONV * 32, qt = ct & 3, e0 = ct >> 2, cw = wid - DP_W_CONV;
        // The two quarters of a 64-channel half write their four 16-byte pieces one
        // after the other, the other half's begin with the third, so that eight lanes
        // write to distinct banks; the codes are loaded in that order.
        const int rot = qt >> 1;
        auto mine = [&](int i) { return STEP * (i + 1) <= DP_KEYS || STEP * i + 8 * cw < DP_KEYS; };  // (the same in a warp)
        uint32_t off[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            off[i] = (uint32_t)rot * DP_HALF + (uint32_t)e0 * 128u + ((((qt & 1) * 4 + ((i + 2 * rot) & 3)) ^ (e0 & 7)) << 4);
        const uint32_t pick0 = rot ? 0x3232u : 0x1010u, pick1 = rot ? 0x1010u : 0x3232u;
        Walk w;
        w.start(a, misc + 2);
        struct Row {
            uint2 k[2], v[2];  // codes of the quarter, in writing order (zeros: not there)
            uint32_t ks, vs;   // its two scales
        };
        auto fetch = [&](uint32_t t, Row (&R)[ENT], uint32_t& missing) {
            missing = 0;
            const int32_t* pages = a.cache.page_table + (int64_t)w.b * a.cache.max_pages_per_seq;
            const int pos0 = (int)(t - w.t0) * DP_KEYS + e0;
#pragma unroll
            for (int i = 0; i < ENT; ++i) {
                const int pos = pos0 + STEP * i;
                R[i].k[0] = R[i].k[1] = R[i].v[0] = R[i].v[1] = make_uint2(0, 0);
                R[i].ks = R[i].vs = 0;
                if (mine(i) && pos < w.seen) {  // (what no token of the unit sees stays unread, its page with it)
                    const int32_t pg = __ldg(pages + (pos >> a.page_shift));
                    if (pg >= 0 && pg < a.cache.n_phys_pages) {
                        const int slot = (pg << a.page_shift) | (pos & ((1 << a.page_shift) - 1));
                        const uint8_t* c = a.cache.codes + (int64_t)slot * kCodeBytes + 16 * qt;
                        const uint8_t* s = a.cache.scales + (int64_t)slot * kScales + 2 * qt;
                        R[i].k[0] = __ldg(reinterpret_cast<const uint2*>(c + 8 * rot));
                        R[i].k[1] = __ldg(reinterpret_cast<const uint2*>(c + 8 * (rot ^ 1)));
                        R[i].v[0] = __ldg(reinterpret_cast<const uint2*>(c + 64 + 8 * rot));
                        R[i].v[1] = __ldg(reinterpret_cast<const uint2*>(c + 64 + 8 * (rot ^ 1)));
                        R[i].ks = __ldg(reinterpret_cast<const uint16_t*>(s));
                        R[i].vs = __ldg(reinterpret_cast<const uint16_t*>(s + 8));
                    } else {
                        dev_error(a.err, CSA2_DEV_PAGE);
                        missing |= 1u << i;
                    }
                }
            }
        };
        // 32 channels of one entry with two scales into a tile
        auto store = [&](uint8_t* tile, const uint2 (&c)[2], uint32_t b2) {
            const uint32_t s2 = e4m3x2_to_h2(b2), s0 = __byte_perm(s2, 0u, pick0), s1 = __byte_perm(s2, 0u, pick1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t sc = i < 2 ? s0 : s1;
                uint32_t h0, h1, h2, h3;
                e2m1x8_to_h2x4(i == 0 ? c[0].x : i == 1 ? c[0].y : i == 2 ? c[1].x : c[1].y, h0, h1, h2, h3);
                *reinterpret_cast<uint4*>(tile + off[i]) = make_uint4(hmul2(h0, sc), hmul2(h1, sc), hmul2(h2, sc), hmul2(h3, sc));
            }
        };
        uint32_t n = 0;  // tiles so far
        Row R[ENT];
        uint32_t missing, t = lo, end;
        bool some = w.tiles(a, t, hi, end);
        if (some) fetch(t, R, missing);
        for (; some; ++n) {
            const int s = (int)(n & 1u);
            // A NaN scale of V may not meet a weight of 0 in the product: V becomes 0 there
            // and K NaN, so the tokens that see the entry get NaN and no other.
            auto nan_pair = [](uint32_t x) { return ((x & 0x7f7fu) + 0x0101u) & 0x8080u; };
            uint32_t nan = 0;
#pragma unroll
            for (int i = 0; i < ENT; ++i) nan |= nan_pair(R[i].vs);
            if (__any_sync(0xffffffffu, nan)) {
#pragma unroll
                for (int i = 0; i < ENT; ++i) {
                    uint32_t x = nan_pair(R[i].vs);
                    R[i].vs &= ~(x | (x - (x >> 7)));  // 0x80 of a byte -> 0xff
                    x |= __shfl_xor_sync(0xffffffffu, x, 1);
                    x |= __shfl_xor_sync(0xffffffffu, x, 2);
                    if (x) R[i].ks = 0x7f7fu;
                }
            }
            if (n >= 2) wait(&kempty[s], ((n >> 1) - 1) & 1u);
            uint8_t* kt = smem + DP_OFF_K + (size_t)s * DP_TILE;
#pragma unroll
            for (int i = 0; i < ENT; ++i)
                if (mine(i)) store(kt + STEP * 128 * i, R[i].k, R[i].ks);
            // which entries are there, one bit each (lane 4 x: entry x of the warp's eight)
#pragma unroll
            for (int i = 0; i < ENT; ++i) {
                uint32_t m = __ballot_sync(0xffffffffu, !((missing >> i) & 1u)) & 0x11111111u;
                m = (m | m >> 3) & 0x03030303u;
                m = (m | m >> 6) & 0x000f000fu;
                m = (m | m >> 12) & 0xffu;
                if (lane == 0 && mine(i)) smem[DP_OFF_OK + (n & 3u) * 16 + STEP / 8 * i + cw] = (uint8_t)m;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kfull[s]);
            uint2 vcode[ENT][2];
            uint32_t vscale[ENT];
#pragma unroll
            for (int i = 0; i < ENT; ++i) {
                vcode[i][0] = R[i].v[0];
                vcode[i][1] = R[i].v[1];
                vscale[i] = R[i].vs;
            }
            ++t;  // the next tile's rows, in flight while V is converted
            some = w.tiles(a, t, hi, end);
            if (some) fetch(t, R, missing);
            if (n >= 2) wait(&vempty[s], ((n >> 1) - 1) & 1u);
            uint8_t* vt = smem + DP_OFF_V + (size_t)s * DP_TILE;
#pragma unroll
            for (int i = 0; i < ENT; ++i)
                if (mine(i)) store(vt + STEP * 128 * i, vcode[i], vscale[i]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&vfull[s]);
        }
    } else if (lo < hi) {
        // ================= softmax and results: row r of row tile i =================
        const int i = wid >> 2, r = (wid & 3) * 32 + lane;
        const uint32_t tS = tmem + ((uint32_t)((wid & 3) * 32) << 16) + 128u * i, tO = tS + 256u;
        Walk w;
        w.start(a, misc + 2);
        uint32_t sn = 0, units = 0, n = 0;  // S tiles and units of this row tile, tiles of the CTA
        if (tid == 0) {
            d.cut[2 * blockIdx.x] = lo > w.t0 && lo < w.te ? make_int4(w.s.row0 + w.k * DP_TOK, w.tokens(), (int)w.t0, (int)w.te)
                                                           : make_int4(-1, 0, 0, 0);
            d.cut[2 * blockIdx.x + 1] = make_int4((int)lo, 0, 0, 0);
        }
        for (uint32_t t = lo, end; w.tiles(a, t, hi, end);) {
            const uint32_t first = t;
            const bool split = w.split<PAIRED>(t, end);
            const int qi = split ? 0 : i, ntok = w.tokens(), tok = 8 * qi + (r >> 4);
            if (8 * qi < ntok) {
                const bool real = tok < ntok;
                const int64_t row = ((int64_t)w.s.row0 + w.k * DP_TOK + tok) * kH + (r & 15);
                const int seen = real ? seen_by(a, w.s, w.k * DP_TOK + tok) : 0;
                // ---- Q: this row, scaled to fp16 ----------------------------------------------
                float c = 1.f;
                {
                    const uint4* q = reinterpret_cast<const uint4*>(a.q + row * kD);
                    uint4 v[4][4];
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[x >> 2][x & 3] = real ? __ldg(q + x) : make_uint4(0, 0, 0, 0);
                    float f;
                    q_scale(fmaxf(fmaxf(q_absmax(v[0]), q_absmax(v[1])), fmaxf(q_absmax(v[2]), q_absmax(v[3]))), f, c);
                    GroupBar{1 + i, 128}.sync();  // the last unit's rows have left the row tile's Q
                    uint8_t* dst = smem + DP_OFF_Q + (size_t)qi * DP_TILE + r * 128;
                    const bool mine = !split || i == 0;  // (the other group only needs c)
#pragma unroll
                    for (int x = 0; x < 16 && mine; ++x) {
                        const uint4 u = v[x >> 2][x & 3];
                        *reinterpret_cast<uint4*>(dst + (size_t)(x >> 3) * DP_HALF + (((x & 7) ^ (r & 7)) << 4)) =
                            make_uint4(q_half2(u.x, f), q_half2(u.y, f), q_half2(u.z, f), q_half2(u.w, f));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && mine) mbar_arrive(&qfull[i]);
                }
                float m = -INFINITY, bias = kPBias, l = 0.f;
                float m_sum = -INFINITY;
                bool drained = false;
                float4* const sums = d.sums + ((size_t)(2 * blockIdx.x + i) * 32) * 128 + r;
                const uint32_t step = split ? 2u : 1u, n_end = n + (end - t);
                if (split) {
                    t += (uint32_t)i;
                    n += (uint32_t)i;
                }
                // O moves to the sums; it is complete, since S of the tile at t is and was issued after O's last product
                auto move_out = [&]() {
                    const float f = m_sum == -INFINITY ? 0.f : ex2(m_sum - m);
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) {
                        uint32_t v[32];
                        tmem_ld32(tO + 32u * x, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float4 u = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                                   __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
                            float4* at = sums + (8 * x + e) * 128;
                            if (drained) {
                                const float4 z = *at;
                                u = make_float4(fmaf(z.x, f, u.x), fmaf(z.y, f, u.y), fmaf(z.z, f, u.z), fmaf(z.w, f, u.w));
                            }
                            *at = u;
                        }
                    }
                    drained = true;
                    m_sum = m;
                    __syncwarp();
                };
                for (;;) {  // runs of tiles: an fp32 result moves O out inside them, a bf16 one between them
                    const uint32_t stop = SPLIT ? end : min(end, t + step * dp_drain(SPLIT));
                    for (; t < stop; t += step, n += step, ++sn) {
                        wait(&sfull[i], sn & 1u);
                        tc_fence_after();
                        if (SPLIT && t - first >= step && ((t - first) / step) % dp_drain(SPLIT) == 0) move_out();
                        else if (SPLIT && t - first >= step) {  // the tile's low terms come on top of kLoScale * O
#pragma unroll 1
                            for (int x = 0; x < 4; ++x) {
                                uint32_t v[32];
                                tmem_ld32(tO + 32u * x, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * kLoScale);
                                tmem_st32(tO + 32u * x, v);
                            }
                        }
                        const int nv = seen - (int)(t - w.t0) * DP_KEYS;  // entries of the tile this row sees
                        const uint4 ok = *reinterpret_cast<const uint4*>(smem + DP_OFF_OK + (n & 3u) * 16);
                        const bool all = __all_sync(0xffffffffu, nv >= DP_KEYS && (ok.x & ok.y & ok.z & ok.w) == ~0u);
                        // ---- 64 columns at a time: maximum, P over S, the sum ---------------------------------
#pragma unroll 1
                        for (int x = 0; x < 2; ++x) {
                            uint32_t v[64];
                            tmem_ld64(tS + 64u * x, v);
                            tmem_wait_ld();
                            if (!all) {  // the columns that this row sees, one bit each
                                const int k = nv - 64 * x;
                                uint64_t b = k >= 64 ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1ull;
                                b &= x == 0 ? (uint64_t)ok.x | (uint64_t)ok.y << 32 : (uint64_t)ok.z | (uint64_t)ok.w << 32;
#pragma unroll
                                for (int e = 0; e < 64; ++e)
                                    if (!((b >> e) & 1u)) v[e] = 0xff800000u;
                            }
                            float mx[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(__uint_as_float(v[e]), __uint_as_float(v[e + 4]));
#pragma unroll
                            for (int e = 8; e < 64; e += 8)
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    mx[y] = fmaxf(fmaxf(mx[y], __uint_as_float(v[e + y])), __uint_as_float(v[e + y + 4]));
                            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;  // log2 domain
                            const bool rise = top > -INFINITY && (m == -INFINITY || top + bias > kPMax);
                            if (__any_sync(0xffffffffu, rise)) {
                                // m takes whole numbers, so O, the sum and P of the tile's earlier columns are
                                // rescaled by a power of two, exactly
                                const float mn = ceilf(top), f = rise && m != -INFINITY ? ex2(m - mn) : 1.f;
                                if (rise) {
                                    m = mn;
                                    bias = kPBias - mn;
                                    l *= f;
                                }
                                __syncwarp();
                                // f as two fp16 factors: it may lie below fp16's range where P times f does not
                                const float fa = fmaxf(f, 0x1p-20f), fb = f / fa;
                                const uint32_t ha = f2_to_h2(fa, fa), hb = f2_to_h2(fb, fb);
                                tmem_wait_st();  // what was stored above is read back: the earlier columns' P (and O)
                                if (x == 1) {
#pragma unroll 1
                                    for (int y = 0; y < 64; y += SPLIT ? 32 : 16) {
                                        uint32_t p[16], q[16];
                                        tmem_ld16(tS + y, p);
                                        if (SPLIT) tmem_ld16(tS + y + 16, q);
                                        tmem_wait_ld();
#pragma unroll
                                        for (int e = 0; e < 16; ++e) {
                                            if (SPLIT) {  // put together, rescaled and taken apart again
                                                const float lo = (h2_lo(p[e]) + h2_lo(q[e]) * (1.f / kLoScale)) * f;
                                                const float hi = (h2_hi(p[e]) + h2_hi(q[e]) * (1.f / kLoScale)) * f;
                                                p[e] = f2_to_h2(lo, hi);
                                                q[e] = rest_h2(lo, hi, p[e]);
                                            } else {
                                                p[e] = hmul2(hmul2(p[e], ha), hb);
                                            }
                                        }
                                        tmem_st16(tS + y, p);
                                        if (SPLIT) tmem_st16(tS + y + 16, q);
                                    }
                                }
                                if (t - first >= step) {  // O is complete: S of this tile was issued after its last product
#pragma unroll 1
                                    for (int y = 0; y < 128; y += 16) {
                                        uint32_t o[16];
                                        tmem_ld16(tO + y, o);
                                        tmem_wait_ld();
#pragma unroll
                                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                        tmem_st16(tO + y, o);
                                    }
                                }
                                tmem_wait_st();
                            }
                            // two columns per packed operation
                            const uint64_t cc = pack_f32x2(c, c), bb = pack_f32x2(bias, bias);
                            uint64_t s0 = 0, s1 = 0;
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                uint32_t p[16], q[16];
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    float p0, p1;
                                    unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[32 * g + e]), __uint_as_float(v[32 * g + e + 1])), cc, bb),
                                                 p0, p1);
                                    p0 = ex2(p0);
                                    p1 = ex2(p1);
                                    if (e & 2) s1 = add_f32x2(s1, pack_f32x2(p0, p1));
                                    else s0 = add_f32x2(s0, pack_f32x2(p0, p1));
                                    p[e >> 1] = f2_to_h2(p0, p1);
                                    if (SPLIT) q[e >> 1] = rest_h2(p0, p1, p[e >> 1]);
                                }
                                tmem_st16(tS + 64u * x + 32u * g, p);
                                if (SPLIT) tmem_st16(tS + 64u * x + 32u * g + 16u, q);
                            }
                            float l0, l1;
                            unpack_f32x2(add_f32x2(s0, s1), l0, l1);
                            l += l0 + l1;
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&pfull[i]);
                    }
                    if (SPLIT || t >= end) break;
                    wait(&sfull[i], sn & 1u);
                    tc_fence_after();
                    move_out();
                }
                t = end;
                n = n_end;
                // ---- the unit's rows ---------------------------------------------------------------
                wait(&ofull[i], units & 1u);
                ++units;
                tc_fence_after();
                const bool whole = first == w.t0 && end == w.te;
                const int64_t part = (2 * (int64_t)blockIdx.x + (first == w.t0 ? 1 : 0)) * DP_ROWS + 128 * qi + r;
                // This thread's piece p (16 bytes) of its row's 64-dim half hf on the way through
                // shared memory: the row tiles' Q, read by now.  8 KiB a warp, 16 where the two
                // groups join (a half each, so that it lies where the second group left its O).
                uint8_t* const stage = smem + DP_OFF_Q + (split ? (size_t)(wid & 3) * 16384 : (size_t)i * DP_TILE + (size_t)(wid & 3) * 8192);
                auto piece_at = [&](int hf, int p) { return reinterpret_cast<uint4*>(stage + (split ? hf * 8192 : 0) + lane * 256 + ((p ^ (lane & 15)) << 4)); };
                float f0 = 1.f, f1 = 0.f;  // factors of this group's O and the other's
                // 32 dims of O from 32 x on, with the sums where O moved there before
                const float f_sum = m_sum == -INFINITY ? 0.f : ex2(m_sum - m);
                auto load_o = [&](int x, uint32_t (&v)[32]) {
                    tmem_ld32(tO + 32u * x, v);
                    tmem_wait_ld();
                    if (drained) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 z = sums[(8 * x + e) * 128];
                            v[4 * e] = __float_as_uint(fmaf(z.x, f_sum, __uint_as_float(v[4 * e])));
                            v[4 * e + 1] = __float_as_uint(fmaf(z.y, f_sum, __uint_as_float(v[4 * e + 1])));
                            v[4 * e + 2] = __float_as_uint(fmaf(z.z, f_sum, __uint_as_float(v[4 * e + 2])));
                            v[4 * e + 3] = __float_as_uint(fmaf(z.w, f_sum, __uint_as_float(v[4 * e + 3])));
                        }
                    }
                };
                if (split) {
                    float2* ml = reinterpret_cast<float2*>(smem + DP_OFF_ML) + r;
                    if (i == 1) {
                        *ml = make_float2(m, l);
#pragma unroll 1
                        for (int x = 0; x < 4; ++x) {
                            uint32_t v[32];
                            load_o(x, v);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *piece_at(x >> 1, 8 * (x & 1) + e) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                        }
                        tc_fence_before();
                    }
                    GroupBar{3, 256}.sync();
                    if (i == 1) {
                        GroupBar{3, 256}.sync();  // the first group has read it, and is done with the row tiles' Q
                        continue;
                    }
                    const float m1 = ml->x, M = fmaxf(m, m1);
                    f0 = m == -INFINITY ? 0.f : ex2(m - M);
                    f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
                    l = (m == -INFINITY ? l : l * f0) + (m1 == -INFINITY ? ml->y : ml->y * f1);  // (a NaN sum stays one)
                    m = M;
                }
                const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
                f0 *= inv;
                f1 *= inv;
                // A row is a thread's, but a store of 32 rows would touch 32 lines: the warp's rows go
                // through its share of the row tile's Q (read by now), 16-byte piece p of a row at
                // p ^ (row & 15), and out 256 bytes of a row at a time.
                const bool bf = whole && a.out_bf16;
                // the warp's first row, and how many of its 32 there are
                const int r0 = (wid & 3) * 32, rows = min(32, max(0, ntok * kH - 128 * qi - r0));
                char* to = whole ? static_cast<char*>(a.out) + (row - lane) * kD * (bf ? 2 : 4)
                                 : reinterpret_cast<char*>(d.part_o + (part - lane) * kD);
#pragma unroll 1
                for (int x = 0; x < 4; ++x) {
                    uint32_t v[32];
                    load_o(x, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f0);
                    if (split) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint4 u = *piece_at(x >> 1, 8 * (x & 1) + e);
                            v[4 * e] = __float_as_uint(fmaf(__uint_as_float(u.x), f1, __uint_as_float(v[4 * e])));
                            v[4 * e + 1] = __float_as_uint(fmaf(__uint_as_float(u.y), f1, __uint_as_float(v[4 * e + 1])));
                            v[4 * e + 2] = __float_as_uint(fmaf(__uint_as_float(u.z), f1, __uint_as_float(v[4 * e + 2])));
                            v[4 * e + 3] = __float_as_uint(fmaf(__uint_as_float(u.w), f1, __uint_as_float(v[4 * e + 3])));
                        }
                    }
                    if (bf) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t y[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[8 * e + 2 * z]), __uint_as_float(v[8 * e + 2 * z + 1]));
                                memcpy(&y[z], &b2, 4);
                            }
                            *piece_at(0, 4 * x + e) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *piece_at(x >> 1, 8 * (x & 1) + e) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                    if (bf ? x == 3 : x & 1) {
                        __syncwarp();
                        const int piece = lane & 15;
                        const int64_t stride = bf ? kD * 2 : kD * 4, at = bf ? 0 : (x >> 1) * 256;
#pragma unroll 4
                        for (int y = lane >> 4; y < rows; y += 2)
                            *reinterpret_cast<uint4*>(to + y * stride + at + piece * 16) =
                                *reinterpret_cast<const uint4*>(stage + (split && !bf ? (x >> 1) * 8192 : 0) + y * 256 + ((piece ^ (y & 15)) << 4));
                        __syncwarp();
                    }
                }
                if (real) {
                    if (whole) {
                        a.lse[row] = l == 0.f ? -INFINITY : (m - kPBias + log2f(l)) * 0.6931471805599453f;
                    } else {
                        d.part_m[part] = m;
                        d.part_l[part] = l;
                    }
                }
                tc_fence_before();
                if (split) GroupBar{3, 256}.sync();
            } else {
                n += end - t;
                t = end;
            }
        }
    } else if (tid == 0) {
        d.cut[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();  // every accumulator has been read
    if (wid == W_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
    if (tid == 0 && *s_timeout) dev_error(a.err, CSA2_DEV_TIMEOUT);
}

// Joins the partial results of every unit that spans CTAs: block (c, y) tokens
// 2 y and 2 y + 1 of the unit that CTA c continues, if CTA c - 1 began it; warp h
// head h of both, sums in a fixed order.  Lane k holds the factors of parts k,
// k + 32, ..., so only the rows themselves are read in the loop, eight at a time.
constexpr int DPJ_THREADS = kH * 32, DPJ_TOK = 2, DPJ_SLOTS = (kDenseCtas + 31) / 32;
__global__ void __launch_bounds__(DPJ_THREADS) dense_prefill_join_kernel(const PrefillDenseArgs d) {
    const int c = blockIdx.x + 1, h = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int4 cut = d.cut[2 * c], at = d.cut[2 * c + 1];
    const int t0 = DPJ_TOK * (int)blockIdx.y;
    if (cut.x < 0 || t0 >= cut.y) return;
    const int per = at.x / c;                 // CTA c begins at place c * per
    if (cut.z < (c - 1) * per) return;        // an earlier CTA's block does it
    const int n = (cut.w - 1) / per - c + 2;  // parts
    auto part = [&](int k, int y) {
        return (int64_t)(k == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + k)) * DP_ROWS + (t0 + y) * kH + h;
    };
    float f[DPJ_TOK][DPJ_SLOTS], M[DPJ_TOK], l[DPJ_TOK];
    float4 o[DPJ_TOK];
#pragma unroll
    for (int y = 0; y < DPJ_TOK; ++y) {  // (a row behind the unit's last holds anything; it is not stored)
        float pl[DPJ_SLOTS];
        M[y] = -INFINITY;
#pragma unroll
        for (int s = 0; s < DPJ_SLOTS; ++s) {
            f[y][s] = lane + 32 * s < n ? d.part_m[part(lane + 32 * s, y)] : -INFINITY;
            pl[s] = lane + 32 * s < n ? d.part_l[part(lane + 32 * s, y)] : 0.f;
            M[y] = fmaxf(M[y], f[y][s]);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) M[y] = fmaxf(M[y], __shfl_xor_sync(0xffffffffu, M[y], s));
        l[y] = 0.f;
#pragma unroll
        for (int s = 0; s < DPJ_SLOTS; ++s) {
            f[y][s] = f[y][s] == -INFINITY ? 0.f : ex2(f[y][s] - M[y]);
            l[y] += pl[s] * f[y][s];
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) l[y] += __shfl_xor_sync(0xffffffffu, l[y], s);
        o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int s = 0; s < DPJ_SLOTS; ++s)
#pragma unroll 8
        for (int k = 32 * s; k < min(n, 32 * s + 32); ++k)
#pragma unroll
            for (int y = 0; y < DPJ_TOK; ++y) {
                const float4 v = *reinterpret_cast<const float4*>(d.part_o + part(k, y) * kD + 4 * lane);
                const float g = __shfl_sync(0xffffffffu, f[y][s], k & 31);
                o[y].x += v.x * g;
                o[y].y += v.y * g;
                o[y].z += v.z * g;
                o[y].w += v.w * g;
            }
#pragma unroll
    for (int y = 0; y < DPJ_TOK; ++y) {
        // eight dims per storing lane
        const float4 u = make_float4(__shfl_down_sync(0xffffffffu, o[y].x, 1), __shfl_down_sync(0xffffffffu, o[y].y, 1),
                                     __shfl_down_sync(0xffffffffu, o[y].z, 1), __shfl_down_sync(0xffffffffu, o[y].w, 1));
        if (!(lane & 1) && t0 + y < cut.y) {
            const float x[8] = {o[y].x, o[y].y, o[y].z, o[y].w, u.x, u.y, u.z, u.w};
            dense_store(d.a, ((int64_t)cut.x + t0 + y) * kH + h, 4 * lane, x, M[y], l[y]);
        }
    }
}

size_t dense_prefill_ws_bytes() {
    return (size_t)2 * kDenseCtas * DP_ROWS * (kD + 2) * 4 + (size_t)2 * kDenseCtas * sizeof(int4) +
           (size_t)kDenseCtas * DP_ROWS * kD * 4;
}

cudaError_t launch_dense_prefill(const DenseArgs& a, char* ws, cudaStream_t stream) {
    static bool init[64];
    static int n_sm[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!init[dev]) {
        for (const void* k : {(const void*)dense_prefill_kernel<false, false>, (const void*)dense_prefill_kernel<true, false>,
                              (const void*)dense_prefill_kernel<false, true>, (const void*)dense_prefill_kernel<true, true>}) {
            e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)DP_SMEM);
            if (e != cudaSuccess) return e;
        }
        e = cudaDeviceGetAttribute(&n_sm[dev], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        init[dev] = true;
    }
    PrefillDenseArgs d{};
    d.a = a;
    d.part_o = reinterpret_cast<float*>(ws);
    d.part_m = d.part_o + (size_t)2 * kDenseCtas * DP_ROWS * kD;
    d.part_l = d.part_m + (size_t)2 * kDenseCtas * DP_ROWS;
    d.cut = reinterpret_cast<int4*>(d.part_l + (size_t)2 * kDenseCtas * DP_ROWS);
    d.sums = reinterpret_cast<float4*>(d.cut + 2 * kDenseCtas);
    // places there can be: units times the longest sequence's tiles and the weight
    const int64_t units = (int64_t)a.T / DP_TOK + a.B, most = units * ((a.max_len + DP_KEYS - 1) / DP_KEYS + DP_WEIGHT);
    const unsigned ctas = (unsigned)std::min<int64_t>(std::min(n_sm[dev], kDenseCtas), most);
    // By the average tokens of a sequence (cu_q is on the device): at most one row
    // tile's take the paired kernel.  Measured, paired / not: 8 x 5 tokens over 65,536
    // entries 69 / 78 us, 8 x 5 over 32,768 45 / 48, 200 x 5 over 400 to 4,000 57 / 62;
    // 4096 tokens over 16,384 entries 534 / 486 us.
    const bool paired = a.T <= DP_TOK / 2 * (int64_t)a.B;
    LaunchCfg c(dim3(ctas), dim3((unsigned)dp_threads(paired)), DP_SMEM, stream);
    auto kernel = a.out_bf16 ? (paired ? dense_prefill_kernel<false, true> : dense_prefill_kernel<false, false>)
                             : (paired ? dense_prefill_kernel<true, true> : dense_prefill_kernel<true, false>);
    e = cudaLaunchKernelEx(&c.cfg, kernel, (const PrefillDenseArgs)d);
    if (e != cudaSuccess || ctas == 1) return e;
    LaunchCfg j(dim3(ctas - 1, DP_TOK / DPJ_TOK), dim3(DPJ_THREADS), 0, stream);
    return cudaLaunchKernelEx(&j.cfg, dense_prefill_join_kernel, (const PrefillDenseArgs)d);
}

}  // namespace csa2

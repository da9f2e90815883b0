// Attention of many queries over compressed caches on tcgen05 tensor cores (sm_100a):
// a prefix that a whole batch shares, read once for all its queries, joined with each
// sequence's own cache (causal inside the residual window for a chunk of new tokens).
//
// For query row i and token t of a block, in the Hadamard domain (q~ = H q, k_hat = H y_t,
// y_t = (u_hat_t s2_t + o) s1_t) with the softmax in log2 units:
//   s_it = q~_i . y_t,   w_it = 2^(s_it - m_i),   out_i = H (sum_t w_it y^v_t) / sum_t w_it.
// A segment is one kv-head of the prefix (rows: every query of the batch that reads that
// head) or one (b, kv-head) of the own caches (rows: its chunk x group).  A tile is one
// 128-token block of a segment, or its residual window, rotated on the way in.  The tiles of
// all (segment, 256-row tile) items form one sequence that is cut into equal ranges, one per
// CTA; a CTA writes the partial (m, l, sum) of each item it touches and a second kernel joins
// them and applies H.
//
// One CTA: 20 warps, three of them idle (registers move between whole warpgroups).
//   warps 8-15  decode tiles into shared memory: a lane gathers codewords (8-fold replicated
//               fp16 codebook, free of bank conflicts), applies signs, scale and mean in fp16,
//               and stores 16-byte chunks of the 128-byte-swizzled operand tile;
//   warp 16     one thread issues the MMAs: S = Q K^T (both from shared memory) into tensor
//               memory and O += P V (P from tensor memory);
//   warps 0-3, 4-7  two softmax groups, each with its own S/P and O columns: a thread owns one
//               query row, so the softmax needs no exchange between lanes.
// With more than 128 rows in an item's tile the groups take 128 rows each and share every K/V
// tile; otherwise both take the same rows and alternate token tiles, as two partials.
//
// Scales: inside a block the fp16 rows are y_t / smax (smax = the largest s1 of the block), so
// they are of order one whatever the norms are; smax of K multiplies the scores, log2 smax of
// V goes into the exponent (so w is scaled by what it contributes, not by what it weighs) and
// its inverse into the denominator.  Rounding to fp16 happens at q~, y and w (2^-11 relative
// at most each); sums, maxima and the denominator are fp32.

#include "hadamard_mma.cuh"
#include "nsn_launch.h"

namespace nsn {
namespace {

constexpr float PF_LOG2E = 1.4426950408889634f;
constexpr float PF_INV_SQRT_D = 0.08838834764831845f;  // 1/sqrt(128)
constexpr int PF_CTAS = 148;       // at most; one per SM
constexpr int PF_DEQ_WARPS = 8;
constexpr int PF_THREADS = 32 * (8 + PF_DEQ_WARPS + 4);  // the last warpgroup: the MMA warp and three idle ones
// Registers per thread after the roles part: at launch all 20 warps hold 96, so the sum over
// the warps may not pass 20 x 96 = 1920: 8 x 120 + 8 x 88 + 4 x 64.
constexpr int PF_REGS_SOFTMAX = 120, PF_REGS_DECODE = 88, PF_REGS_MMA = 64;
static_assert(8 * PF_REGS_SOFTMAX + PF_DEQ_WARPS * PF_REGS_DECODE + 4 * PF_REGS_MMA <= (PF_THREADS / 32) * 96, "registers of the CTA");
constexpr int PF_RING = 3;         // K / V tiles in shared memory
constexpr int PF_TILE_BYTES = 32768;  // 128 tokens (or rows) x 128 dims fp16: two 16 KB halves of 64 dims
constexpr uint32_t PF_HALF = 16384u;
// The running max moves only when a score exceeds it by more than this (log2 units): w stays
// below 2^8, and most tiles leave O alone.
constexpr float PF_SLACK = 8.0f;
constexpr uint32_t PF_WAIT_LIMIT = 1u << 22;   // attempts of a wait before it gives up (seconds)
constexpr uint32_t PF_POLL_LIMIT = 1u << 26;   // idle rounds of the MMA thread's event loop (seconds)

struct RowSet {  // the rows of one kind of segment
  int rows;      // query rows of a segment
  int rt;        // 256-row tiles
  int hr;        // rows of one group's half of a partial slot (128, or the rows rounded up to 32)
};

struct PfArgs {
  CacheView pk, pv, k, v;  // prefix (batch 1) and own caches
  const void* q;
  int dtype;
  int64_t qsb, qst, qsh;
  float qscale;            // softmax scale * log2 e / sqrt(128)
  const float *cbk, *cbv;
  int B, C, H, G;
  int causal;              // own window: query c sees slots up to n_window - C + c
  RowSet rp, ro;
  unsigned char* qt;       // rotated query tiles: two of hr rows per item, prefix items first
  int2* tab;               // per item: first and last CTA
  float2* ml;              // partial (m, l): prefix slots, then own slots
  float* acc;              // partial sums, same slots
  const float* own_out;    // not null: the own part's rows come from the decode kernel (then ro is empty),
  const float2* own_lse;   //   each with its (max in log2 units, denominator)
  int32_t* status;
};

struct PfInfo {            // of one tile, for the softmax
  float ka, lv, iva;       // K scale, log2 and inverse of the V scale
  int nvalid;              // tokens
  int vbad;                // first token whose V row is not finite (128: none)
  int base;                // window tile of a causal segment: query c sees base + c tokens; else nvalid, step 0
  int step;
  int pad;
};

struct PfSmem {
  alignas(1024) unsigned char q[2][PF_TILE_BYTES];
  alignas(1024) unsigned char ring[PF_RING][PF_TILE_BYTES];
  alignas(128) uint4 cbk[NCODES][8];
  alignas(128) uint4 cbv[NCODES][8];
  alignas(16) unsigned char o[PF_DEQ_WARPS][128];  // the half mean row of the tile a decode warp is at
  alignas(16) PfInfo info[4];
  alignas(16) float red[2][PF_DEQ_WARPS];
  int red_bad[PF_DEQ_WARPS];
  alignas(8) uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], full[PF_RING], empty[PF_RING], meet, drain;
  long long scan[PF_THREADS / 32];
  long long units;
  int seg0, rt0, u0;
  uint32_t tmem;
  int fail;
};
static_assert(sizeof(PfSmem) + 1024 <= 232448, "shared memory of one SM");

// ---------------------------------------------------------------------------
// Barriers, tensor core and tensor memory
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t sm_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(sm_addr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(sm_addr(b)) : "memory");
}
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done) : "r"(sm_addr(b)), "r"(parity & 1u) : "memory");
  return done != 0;
}
// Bounded wait; false if it gave up or another role did.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, volatile int* fail) {
  for (uint32_t i = 0; i < PF_WAIT_LIMIT; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(sm_addr(b)), "r"(parity & 1u) : "memory");
    if (done) return true;
    if (*fail) return false;
  }
  return false;
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// (by the elected lane of a converged warp)
__device__ __forceinline__ void tc_commit_to(uint64_t* b) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(sm_addr(b)) : "memory");
}

// Matrix descriptors of the 128-byte-swizzled operands (descriptor version 1, layout 2): 8-row
// groups of 128-byte rows 1024 B apart; the leading offset is the distance of the two 64-dim
// halves where the operand is read across them (V: dims are the N axis).
// kind::f16, fp32 accumulator, fp16 operands, M = N = 128; V is read with its N axis (dims) contiguous.
constexpr uint32_t PF_IDESC_QK = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t PF_IDESC_PV = PF_IDESC_QK | (1u << 16);

// Issued by one elected lane of a converged warp: with the operands uniform across the warp the
// compiler keeps them in uniform registers (about 35 cycles an MMA; from a single-lane branch each
// operand is moved there first, 55 cycles alone and over 100 beside busy warps).  A descriptor is its
// low word (start address and leading offset) and the constant high word.
constexpr uint32_t PF_DESC_HI = (uint32_t)(((1024ull >> 4 << 32) | (1ull << 46) | (2ull << 61)) >> 32);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 da, db;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n"
      ::"r"(d), "r"(a), "r"(b), "r"(PF_IDESC_QK), "r"((uint32_t)accumulate), "r"(PF_DESC_HI) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 db;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 db, {%2, %5};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n"
      ::"r"(d), "r"(a), "r"(b), "r"(PF_IDESC_PV), "r"((uint32_t)accumulate), "r"(PF_DESC_HI) : "memory");
}

// 32 columns of this warp's 32 tensor-memory lanes; to be read only after tm_ready32.
__device__ __forceinline__ void tm_ld32_async(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr) : "memory");
}
__device__ __forceinline__ void tm_ready32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :: "memory");
}
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t (&r)[32]) {
  tm_ld32_async(addr, r);
  tm_ready32(r);
}
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr) : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 values in a register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pack_f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack_f2(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// ---------------------------------------------------------------------------
// Segments, tiles and the pieces of one CTA's range
// ---------------------------------------------------------------------------
struct Seg {
  int nq, nw, blocks, tiles;  // quantized tokens, window tokens, 128-token blocks, tiles
};
__device__ __forceinline__ Seg seg_info(const PfArgs& a, int seg) {
  const bool own = seg >= a.H;
  const CacheView& kc = own ? a.k : a.pk;
  const CacheView& vc = own ? a.v : a.pv;
  const int64_t i = own ? seg - a.H : seg;
  Seg s;
  s.nq = max(0, min(min(__ldg(kc.n_quant + i), __ldg(vc.n_quant + i)), kc.capacity));
  s.nw = kc.window_len > 0 ? max(0, min(min(__ldg(kc.n_window + i), __ldg(vc.n_window + i)), kc.window_len)) : 0;
  s.blocks = (s.nq + BLK - 1) / BLK;
  s.tiles = s.blocks + (s.nw > 0 ? 1 : 0);
  return s;
}

// One item's share of this CTA's range: tiles [j, j + m) of 256-row tile rt of segment seg.
struct Piece {
  int seg, rt, j, m;
  Seg s;
  bool own, dual;   // dual: at most 128 rows, the groups alternate tiles
  int rows;         // rows of the 256-row tile that exist
  int64_t item;     // index among the items of its kind
};
// Ranges are cut in units of one tile plus PF_ITEM_COST for each item (its query operand, the
// latency of its first scores and its partial, which are not overlapped with other items).
constexpr int PF_ITEM_COST = 3;
__device__ __forceinline__ int seg_units(const Seg& s) { return s.tiles > 0 ? s.tiles + PF_ITEM_COST : 0; }
struct Cursor {
  int seg, rt, u;   // unit within the item
  long long left;   // units of this CTA's range
};
__device__ __forceinline__ bool next_piece(const PfArgs& a, Cursor& c, Piece& p) {
  do {
    if (c.left <= 0) return false;
    p.s = seg_info(a, c.seg);
    while (p.s.tiles == 0) p.s = seg_info(a, ++c.seg);  // `left` counts units of existing tiles, so there is one
    p.seg = c.seg;
    p.rt = c.rt;
    p.own = c.seg >= a.H;
    const RowSet& r = p.own ? a.ro : a.rp;
    const int units = seg_units(p.s), n = (int)min((long long)(units - c.u), c.left);
    p.j = max(0, c.u - PF_ITEM_COST);
    p.m = max(0, c.u + n - PF_ITEM_COST) - p.j;
    p.rows = min(256, r.rows - 256 * c.rt);
    p.dual = p.rows <= 128;
    p.item = (int64_t)(p.own ? c.seg - a.H : c.seg) * r.rt + c.rt;
    c.left -= n;
    c.u += n;
    if (c.u == units) {
      c.u = 0;
      if (++c.rt == r.rt) {
        c.rt = 0;
        ++c.seg;
      }
    }
  } while (p.m == 0);  // (the range ended inside the item's overhead)
  return true;
}
// Ring index, from the piece's base, of tile t's K and V: the order is K0 K1 V0 K2 V1 ... V(m-1).
__device__ __forceinline__ int ring_k(int t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int ring_v(int t, int m) { return t + 1 < m ? 2 * t + 2 : 2 * m - 1; }

// Partial slots: a CTA walks the items in order, so (item + CTA) names each (item, CTA) pair
// once; prefix items' slots come first.
__device__ __forceinline__ int64_t slot_row(const PfArgs& a, bool own, int64_t item, int64_t cta) {
  if (!own) return (item + cta) * 2 * a.rp.hr;
  return ((int64_t)a.H * a.rp.rt + PF_CTAS) * 2 * a.rp.hr + (item + cta) * 2 * a.ro.hr;
}
// Element c of a slot's row: 8-dim groups of all the slot's rows lie together, so that the
// threads of a warp (32 consecutive rows) write, and a warp of the join reads, whole sectors.
__device__ __forceinline__ int64_t acc_off(int64_t row0, int hr, int row, int c) {
  return row0 * D + ((int64_t)(c >> 3) * (2 * hr) + row) * 8 + (c & 7);
}

// ---------------------------------------------------------------------------
// Decode warps
// ---------------------------------------------------------------------------
// What a lane reads for one K or V tile of a quantized block: token 32 (w >> 1) + lane,
// sub-vectors 8 (w & 1) .. + 7 of it, and what the block's largest s1 needs.
struct Raw {
  uint32_t ce, co;        // codes of the even and odd sub-vectors
  uint4 sign;
  uint32_t norm;          // fp16 (s1, s2), or fp16 s2 and the s1 level
  uint4 four;             // s1 of tokens 4 lane .. 4 lane + 3 (fp16 pairs, or levels)
  uint32_t mean;          // dims 64 (w & 1) + 2 lane, + 1
  uint2 par;              // fp16 (s1 lo, s1 hi, o lo, o hi)
};

// Base addresses of one sequence's quantized buffers.
struct Src {
  const unsigned char *codes, *signs, *norms, *means, *levels, *params;
};
template <bool DQ>
__device__ __forceinline__ Src seq_src(const CacheView& c, int64_t seq) {
  const int64_t t = seq * c.capacity, b = seq * (c.capacity / BLK);
  Src s;
  s.codes = c.codes + t * NSUB;
  s.signs = c.signs + t * NSUB;
  s.norms = reinterpret_cast<const unsigned char*>(c.norms) + t * (DQ ? 2 : 4);
  s.means = reinterpret_cast<const unsigned char*>(c.means) + b * (DQ ? D / 2 : 2 * D);
  s.levels = DQ ? c.s1_levels + t / 2 : nullptr;
  s.params = DQ ? reinterpret_cast<const unsigned char*>(c.dq_params) + b * 16 : nullptr;
  return s;
}

// The s1 of a block's tokens 4 lane .. 4 lane + 3.
template <bool DQ>
__device__ __forceinline__ void four_load(uint4& four, uint2& par, const Src& c, int64_t blk, int lane) {
  if constexpr (DQ) {
    four.x = __ldg(reinterpret_cast<const unsigned short*>(c.levels + blk * (BLK / 2)) + lane);
    par = __ldg(reinterpret_cast<const uint2*>(c.params + blk * 16));
  } else {
    four = __ldg(reinterpret_cast<const uint4*>(c.norms + blk * (4 * BLK)) + lane);
  }
}

template <int MODE, bool DQ>
__device__ __forceinline__ void raw_load(Raw& r, const Src& c, int64_t blk, int w, int lane) {
  const int hs = w & 1, t = 32 * (w >> 1) + lane;
  const uint32_t* code = reinterpret_cast<const uint32_t*>(c.codes + blk * (BLK * NSUB)) + 4 * t;
  r.ce = __ldg(code + hs);
  r.co = __ldg(code + 2 + hs);
  if constexpr (MODE == NSN_MODE_2BIT) r.sign = __ldg(reinterpret_cast<const uint4*>(c.signs + blk * (BLK * NSUB)) + t);
  if constexpr (DQ) {
    const uint32_t lev = (uint32_t)__ldg(c.levels + blk * (BLK / 2) + t / 2) >> (4 * (uint32_t)(t & 1)) & 15u;
    r.norm = (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(c.norms + blk * (2 * BLK)) + t) | (lev << 16);
    r.mean = __ldg(c.means + blk * (D / 2) + 32 * hs + lane);
  } else {
    r.norm = __ldg(reinterpret_cast<const uint32_t*>(c.norms + blk * (4 * BLK)) + t);
    r.mean = __ldg(reinterpret_cast<const uint32_t*>(c.means + blk * (2 * D)) + 32 * hs + lane);
  }
  four_load<DQ>(r.four, r.par, c, blk, lane);
}

__device__ __forceinline__ float2 lo_step(uint32_t lohi) {
  const float2 v = __half22float2(as_h2(lohi));
  return make_float2(v.x, (v.y - v.x) * (1.0f / 15.0f));
}

// Largest |s1| of a block's valid tokens (all lanes).
template <bool DQ>
__device__ __forceinline__ float block_smax(const uint4& four, const uint2& par, int nvalid, int lane) {
  float m = 0.f;
  const uint32_t w[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float s;
    if constexpr (DQ) {
      const float2 ls = lo_step(par.x);
      s = fmaf((float)((four.x >> (4 * i)) & 15u), ls.y, ls.x);
    } else {
      s = __low2float(as_h2(w[i]));
    }
    if (4 * lane + i < nvalid) m = fmaxf(m, fabsf(s));
  }
  return warp_max(m);
}

// Writes this warp's share of a decoded tile: fp16((u_hat s2 + o) s1 / smax) per token.
template <int MODE, bool DQ>
__device__ __forceinline__ void tile_write(const Raw& r, const uint4 (*cb)[8], unsigned char* tile, unsigned char* orow,
                                           float smax, int nvalid, int w, int lane) {
  const int hs = w & 1, row = 32 * (w >> 1) + lane;
  float s1, s2;
  uint32_t mean = r.mean;
  if constexpr (DQ) {
    const float2 ls = lo_step(r.par.x), lo = lo_step(r.par.y);
    s1 = fmaf((float)(r.norm >> 16), ls.y, ls.x);
    s2 = __low2float(as_h2(r.norm));
    mean = pack_h2(fmaf((float)(r.mean & 15u), lo.y, lo.x), fmaf((float)(r.mean >> 4), lo.y, lo.x));
  } else {
    const float2 n = __half22float2(as_h2(r.norm));
    s1 = n.x;
    s2 = n.y;
  }
  const float ratio = smax > 0.f ? s1 / smax : 0.f;
  const __half2 b2 = __float2half2_rn(ratio), a2 = __float2half2_rn(ratio * s2);
  __syncwarp();  // the previous tile's mean row has been read
  reinterpret_cast<uint32_t*>(orow)[lane] = mean;
  __syncwarp();
  unsigned char* dst = tile + hs * PF_HALF + row * 128;
  const bool live = row < nvalid;
  const uint4* rep = &cb[0][lane & 7];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t code = __byte_perm((k & 1) ? r.co : r.ce, 0u, 0x4440u | (uint32_t)(k >> 1));
    const uint4 c = rep[code * 8];
    const uint4 o = *reinterpret_cast<const uint4*>(orow + 16 * k);
    uint32_t u[4] = {c.x, c.y, c.z, c.w};
    const uint32_t om[4] = {o.x, o.y, o.z, o.w};
    if constexpr (MODE == NSN_MODE_2BIT) {
      const uint32_t sw[4] = {r.sign.x, r.sign.y, r.sign.z, r.sign.w};
      const int s = 8 * hs + k;  // the sign of dim 8 s + i is bit 15 - s of field i
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] ^= (sw[i] << s) & 0x80008000u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = as_u32(__hfma2(as_h2(u[i]), a2, __hmul2(as_h2(om[i]), b2)));
    *reinterpret_cast<uint4*>(dst + ((k ^ (row & 7)) << 4)) =
        live ? make_uint4(u[0], u[1], u[2], u[3]) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// Window rows 16 w .. 16 w + 15 of one sequence as A fragments of the transform (rows past nw: zero).
__device__ __forceinline__ void window_load(uint32_t (&f)[8][4], const CacheView& c, int64_t seq, int nw, int w, int lane) {
  const int g = lane >> 2, p = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 16 * w + g + 8 * i;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(c.window + (seq * c.window_len + t) * (int64_t)D) + p;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      f[r][i] = t < nw ? __ldg(row + 8 * r) : 0u;
      f[r][2 + i] = t < nw ? __ldg(row + 8 * r + 4) : 0u;
    }
  }
}

// The largest root mean square of those rows that are finite, and the first row that is not.
__device__ __forceinline__ void window_scan(const uint32_t (&f)[8][4], int w, int lane, float& smax, int& bad) {
  smax = 0.f;
  bad = BLK;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float ss = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float2 x = __half22float2(as_h2(f[r][i])), y = __half22float2(as_h2(f[r][2 + i]));
      ss += x.x * x.x + x.y * x.y + y.x * y.x + y.y * y.y;
    }
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    if (ss <= 3.0e38f) smax = fmaxf(smax, sqrtf(ss * (1.0f / D)));
    else bad = min(bad, 16 * w + (lane >> 2) + 8 * i);
  }
  smax = warp_max(smax);
  bad = __reduce_min_sync(0xffffffffu, bad);
}

// Four consecutive dims 16 r + 4 p of row t of an operand tile, as fp16 (`half`: bytes between its 64-dim halves).
__device__ __forceinline__ void put4(unsigned char* tile, int64_t half, int t, int r, int p, float a, float b, float c, float d) {
  const int chunk = 2 * r + (p >> 1);
  unsigned char* dst = tile + (chunk >> 3) * half + t * 128 + (((chunk & 7) ^ (t & 7)) << 4) + (p & 1) * 8;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_h2(a, b), pack_h2(c, d));
}

// Writes those rows rotated, fp16(H x / smax); rows that are not finite are zero where `drop`
// (V: a zero weight would not cancel them).
__device__ __forceinline__ void window_write(const uint32_t (&f)[8][4], float smax, bool drop, unsigned char* tile, int w, int lane) {
  uint32_t hb[2][2];
  h16_operand(hb, lane);
  float E[8][2][4];
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      E[r][nt][0] = E[r][nt][1] = E[r][nt][2] = E[r][nt][3] = 0.f;
      h16_mma(E[r][nt], f[r], hb[nt]);
    }
  h8_butterflies(E);
  const float inv = smax > 0.f ? PF_INV_SQRT_D / smax : 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // an element that is not finite reaches every element of its row
    const bool zero = drop && !(fabsf(E[0][0][2 * i]) <= 3.0e38f);
#pragma unroll
    for (int r = 0; r < 8; ++r)
      put4(tile, PF_HALF, 16 * w + (lane >> 2) + 8 * i, r, lane & 3, zero ? 0.f : E[r][0][2 * i] * inv, zero ? 0.f : E[r][0][2 * i + 1] * inv,
           zero ? 0.f : E[r][1][2 * i] * inv, zero ? 0.f : E[r][1][2 * i + 1] * inv);
  }
}

// Meets the other decode warps (bounded, as every wait here); `phase` counts the meetings.
__device__ __forceinline__ bool decode_sync(PfSmem& sm, uint32_t& phase, int lane) {
  __syncwarp();
  if (lane == 0) bar_arrive(&sm.meet);
  return bar_wait(&sm.meet, phase++, &sm.fail);
}

// One decode warp's walk over the pieces: tasks in ring order, the next task's global reads
// issued before the current one waits for its slot.
template <int MK, int MV, bool DQ>
__device__ __forceinline__ bool decode_role(const PfArgs& a, PfSmem& sm, Cursor cur, int w, int lane) {
  Piece p;
  int n = 0;  // ring index
  uint32_t met = 0;
  float window_vmax = 0.f;  // V scale of the piece's window tile
  while (next_piece(a, cur, p)) {
    const CacheView& kc = p.own ? a.k : a.pk;
    const CacheView& vc = p.own ? a.v : a.pv;
    const int64_t seq = p.own ? p.seg - a.H : p.seg;
    const Src ks = seq_src<DQ>(kc, seq), vs = seq_src<DQ>(vc, seq);
    const int base = n, tasks = 2 * p.m;
    Raw next, vraw;
    uint4 v4 = make_uint4(0u, 0u, 0u, 0u);   // V norms of a K task's block (for the tile's scales)
    uint2 vp = make_uint2(0u, 0u);
    // task i of the piece: K of tile (i + 1) / 2 for odd i and i = 0, V of tile i / 2 - 1 for even i, V of the last tile at the end
    const auto is_k = [&](int i) { return i == 0 || ((i & 1) && i != tasks - 1); };
    const auto tile_of = [&](int i) { return i == 0 ? 0 : i == tasks - 1 ? p.m - 1 : (i & 1) ? (i + 1) / 2 : i / 2 - 1; };
    const auto fetch = [&](int i) {
      const int blk = p.j + tile_of(i);
      if (blk >= p.s.blocks) return;
      if (is_k(i)) {
        raw_load<MK, DQ>(next, ks, blk, w, lane);
        four_load<DQ>(v4, vp, vs, blk, lane);
      } else {
        raw_load<MV, DQ>(next, vs, blk, w, lane);
      }
    };
    fetch(0);
    for (int i = 0; i < tasks; ++i, ++n) {
      vraw = next;
      const uint4 c4 = v4;
      const uint2 cp = vp;
      if (i + 1 < tasks) fetch(i + 1);
      const int t = tile_of(i), blk = p.j + t, slot = n % PF_RING;
      const bool k_task = is_k(i);
      if (n >= PF_RING && !bar_wait(&sm.empty[slot], (uint32_t)(n / PF_RING - 1), &sm.fail)) return false;
      unsigned char* tile = sm.ring[slot];
      PfInfo info;
      if (blk < p.s.blocks) {
        const int nvalid = min(BLK, p.s.nq - BLK * blk);
        const float smax = block_smax<DQ>(vraw.four, vraw.par, nvalid, lane);
        if (k_task) {
          tile_write<MK, DQ>(vraw, sm.cbk, tile, sm.o[w], smax, nvalid, w, lane);
          const float vmax = block_smax<DQ>(c4, cp, nvalid, lane);
          info.ka = smax > 0.f ? smax : 1.f;
          info.iva = vmax > 0.f ? vmax : 1.f;
          info.vbad = BLK;
          info.nvalid = info.base = nvalid;
          info.step = 0;
        } else {
          tile_write<MV, DQ>(vraw, sm.cbv, tile, sm.o[w], smax, nvalid, w, lane);
        }
      } else {
        float smax = window_vmax;
        int vbad = BLK;
        uint32_t f[8][4];
        if (k_task) {  // scales of K and V over the whole tile (V is read again for its own task)
          float mine, mine_v;
          int bad;
          window_load(f, vc, seq, p.s.nw, w, lane);
          window_scan(f, w, lane, mine_v, vbad);
          window_load(f, kc, seq, p.s.nw, w, lane);
          window_scan(f, w, lane, mine, bad);
          if (lane == 0) {
            sm.red[0][w] = mine;
            sm.red[1][w] = mine_v;
            sm.red_bad[w] = vbad;
          }
          if (!decode_sync(sm, met, lane)) return false;
          smax = window_vmax = 0.f;
#pragma unroll
          for (int x = 0; x < PF_DEQ_WARPS; ++x) {
            smax = fmaxf(smax, sm.red[0][x]);
            window_vmax = fmaxf(window_vmax, sm.red[1][x]);
            vbad = min(vbad, sm.red_bad[x]);
          }
          if (!decode_sync(sm, met, lane)) return false;
        } else {
          window_load(f, vc, seq, p.s.nw, w, lane);
        }
        window_write(f, smax, !k_task, tile, w, lane);
        const float vmax = window_vmax;
        info.ka = smax > 0.f ? smax : 1.f;
        info.iva = vmax > 0.f ? vmax : 1.f;
        info.vbad = vbad;
        info.nvalid = p.s.nw;
        info.step = p.own && a.causal ? 1 : 0;
        info.base = info.step ? p.s.nw - a.C + 1 : p.s.nw;
      }
      if (k_task && w == 0 && lane == 0) {
        info.lv = log2f(info.iva);
        info.iva = 1.f / info.iva;
        sm.info[(base / 2 + t) & 3] = info;
      }
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(&sm.full[slot]);
    }
  }
  return true;
}

// ---------------------------------------------------------------------------
// The MMA warp: an event loop over the two groups of a piece.  A group alternates
// S = Q K^T of a tile (needs the K tile, and its previous P consumed) and O += P V (needs the
// V tile and P); whichever group can go, goes.  The warp stays converged (votes decide).
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool test_all(uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, bar_test(b, parity)); }

struct MmaGroup {
  int t;           // tile it is at
  bool pv, first;  // waiting for P; no tile of the piece finished yet
  uint32_t done;   // tiles finished, over all pieces
  uint32_t built;  // query operands used, over all pieces
};

// One step of group I if it can go.
template <int I>
__device__ __forceinline__ bool mma_step(PfSmem& sm, MmaGroup& s, const Piece& p, int n0, uint32_t tmem, uint32_t q_lo, uint32_t k_lo, uint32_t v_lo) {
  if (s.t >= p.m) return false;
  const uint32_t s_col = tmem + 128u * I, o_col = tmem + 256u + 128u * I;
  constexpr uint32_t TILE = PF_TILE_BYTES >> 4;
  if (!s.pv) {
    const int n = n0 + ring_k(s.t), slot = n % PF_RING;
    if (s.first ? !test_all(&sm.q_full[I], s.built) : !test_all(&sm.pv_done[I], s.done - 1u)) return false;
    if (!test_all(&sm.full[slot], (uint32_t)(n / PF_RING))) return false;
    tc_after();
    const uint32_t kd = k_lo + TILE * (uint32_t)slot;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t step = ((k >> 2) * PF_HALF + (k & 3) * 32u) >> 4;
      mma_ss(s_col, q_lo + TILE * I + step, kd + step, k > 0);
    }
    tc_commit_to(&sm.s_full[I]);
    tc_commit_to(&sm.empty[slot]);
    if (p.dual) tc_commit_to(&sm.empty[slot]);  // the barrier counts both groups
    s.pv = true;
  } else {
    const int n = n0 + ring_v(s.t, p.m), slot = n % PF_RING;
    if (!test_all(&sm.p_full[I], s.done)) return false;
    if (!test_all(&sm.full[slot], (uint32_t)(n / PF_RING))) return false;
    tc_after();
    const uint32_t vd = v_lo + TILE * (uint32_t)slot;
#pragma unroll
    for (int k = 0; k < 8; ++k) mma_ts(o_col, s_col + 8u * k, vd + 128u * k, !s.first || k > 0);
    tc_commit_to(&sm.pv_done[I]);
    tc_commit_to(&sm.empty[slot]);
    if (p.dual) tc_commit_to(&sm.empty[slot]);
    s.pv = s.first = false;
    ++s.done;
    s.t += p.dual ? 2 : 1;
  }
  return true;
}

__device__ __forceinline__ bool mma_role(const PfArgs& a, PfSmem& sm, Cursor cur) {
  // descriptors differ from these only by constant steps of the start address (16-byte units)
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
  const uint32_t q_lo = desc_lo(sm_addr(sm.q[0]), 16u), k_lo = desc_lo(sm_addr(sm.ring[0]), 16u), v_lo = desc_lo(sm_addr(sm.ring[0]), PF_HALF);
  Piece p;
  int n0 = 0;
  MmaGroup g0 = {0, false, true, 0u, 0u}, g1 = g0;
  while (next_piece(a, cur, p)) {
    p.m = __shfl_sync(0xffffffffu, p.m, 0);
    p.dual = __all_sync(0xffffffffu, p.dual);
    g0.t = 0;
    g1.t = p.dual ? 1 : 0;
    g0.pv = g1.pv = false;
    g0.first = g1.first = true;
    uint32_t idle = 0;
    while (g0.t < p.m || g1.t < p.m) {
      const bool m0 = mma_step<0>(sm, g0, p, n0, tmem, q_lo, k_lo, v_lo);
      const bool m1 = mma_step<1>(sm, g1, p, n0, tmem, q_lo, k_lo, v_lo);
      if (m0 || m1) idle = 0;
      else if (++idle > PF_POLL_LIMIT || ((idle & 255u) == 0u && __any_sync(0xffffffffu, *(volatile int*)&sm.fail))) return false;
    }
    // (a group without tiles here - one tile, alternating groups - has not built a query operand)
    g0.built += g0.first ? 0u : 1u;
    g1.built += g1.first ? 0u : 1u;
    n0 += 2 * p.m;
  }
  return true;
}

// ---------------------------------------------------------------------------
// Queries: H q in log2 units, fp16, laid out as the operand tiles that prefix_kernel copies whole
// (once per row here, instead of once per row and CTA there).  One warp takes 16 rows of an item.
// ---------------------------------------------------------------------------
// Query of row `row` of an item (its 256-row tile rt): batch, chunk position, head.
struct RowAt { int b, c, h; };
__device__ __forceinline__ RowAt row_at(const PfArgs& a, bool own, int seg, int row) {
  RowAt r;
  const int per = a.C * a.G;
  const int seq = seg - a.H;
  const int in = own ? row : row % per;
  r.b = own ? seq / a.H : row / per;
  r.c = in / a.G;
  r.h = (own ? seq % a.H : seg) * a.G + in % a.G;
  return r;
}

// The A fragments (fp16 hi + lo) of r of 16 query rows, from this lane's raw reads.
template <int DT>
__device__ __forceinline__ void q_split(const uint2 (&x)[2][2], float scale, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      float2 v;
      if constexpr (DT == NSN_DTYPE_F32) v = make_float2(__uint_as_float(x[i][kk].x), __uint_as_float(x[i][kk].y));
      else if constexpr (DT == NSN_DTYPE_BF16) v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[i][kk].x));
      else v = __half22float2(as_h2(x[i][kk].x));
      split_half2(v.x * scale, v.y * scale, hi[2 * kk + i], lo[2 * kk + i]);
    }
}
template <int DT>
__device__ __forceinline__ void q_transform(float (&E)[8][2][4], const void* q, float scale, const int64_t (&off)[2],
                                            const bool (&have)[2], const uint32_t (&hb)[2][2]) {
  constexpr int RN = DT == NSN_DTYPE_F32 ? 4 : 8;  // r's read at once (32 registers)
#pragma unroll
  for (int r0 = 0; r0 < 8; r0 += RN) {
    uint2 x[RN][2][2];
#pragma unroll
    for (int r = 0; r < RN; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const int64_t o = off[i] + 16 * (r0 + r) + 8 * kk;
          x[r][i][kk] = make_uint2(0u, 0u);
          if (have[i]) {
            if constexpr (DT == NSN_DTYPE_F32) x[r][i][kk] = __ldg(reinterpret_cast<const uint2*>(static_cast<const float*>(q) + o));
            else x[r][i][kk].x = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(q) + o));
          }
        }
#pragma unroll
    for (int r = 0; r < RN; ++r) {
      uint32_t hi[4], lo[4];
      q_split<DT>(x[r], scale, hi, lo);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float(&e)[4] = E[r0 + r][nt];
        e[0] = e[1] = e[2] = e[3] = 0.f;
        h16_mma(e, hi, hb[nt]);
        h16_mma(e, lo, hb[nt]);
      }
    }
  }
  h8_butterflies(E);
}

constexpr int QUERY_WARPS = 4;

// Bytes of one hr-row tile, and the tile of an item's group.
__device__ __host__ __forceinline__ int64_t q_tile_bytes(const RowSet& r) { return (int64_t)r.hr * 2 * D; }
__device__ __forceinline__ unsigned char* q_tile(const PfArgs& a, bool own, int64_t item, int group) {
  return own ? a.qt + (int64_t)a.H * a.rp.rt * 2 * q_tile_bytes(a.rp) + (item * 2 + group) * q_tile_bytes(a.ro)
             : a.qt + (item * 2 + group) * q_tile_bytes(a.rp);
}

__global__ void __launch_bounds__(32 * QUERY_WARPS) prefix_query_kernel(const __grid_constant__ PfArgs a) {
  const int lane = threadIdx.x & 31, g = lane >> 2, pr = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t unit = (int64_t)blockIdx.x * QUERY_WARPS + (threadIdx.x >> 5);
  const int np = (a.rp.rows + 15) / 16, no = (a.ro.rows + 15) / 16;  // 16-row groups of a segment
  const bool own = unit >= (int64_t)a.H * np;
  const int64_t u = own ? unit - (int64_t)a.H * np : unit;
  const RowSet& rs = own ? a.ro : a.rp;
  const int per = own ? no : np;
  const int s = per > 0 ? (int)(u / per) : a.B * a.H;   // segment of its kind
  if (s < (own ? a.B * a.H : a.H)) {
    const int row0 = 16 * (int)(u % per);
    int64_t off[2];
    bool have[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + g + 8 * i;
      have[i] = row < rs.rows;
      const RowAt r = row_at(a, own, own ? a.H + s : s, have[i] ? row : row0);
      off[i] = (int64_t)r.b * a.qsb + (int64_t)r.c * a.qst + (int64_t)r.h * a.qsh + 2 * pr;
    }
    uint32_t hb[2][2];
    h16_operand(hb, lane);
    float E[8][2][4];
    if (a.dtype == NSN_DTYPE_F32) q_transform<NSN_DTYPE_F32>(E, a.q, a.qscale, off, have, hb);
    else if (a.dtype == NSN_DTYPE_BF16) q_transform<NSN_DTYPE_BF16>(E, a.q, a.qscale, off, have, hb);
    else q_transform<NSN_DTYPE_F16>(E, a.q, a.qscale, off, have, hb);
    unsigned char* tile = q_tile(a, own, (int64_t)s * rs.rt + row0 / 256, (row0 / 128) & 1);
    const int64_t half = (int64_t)rs.hr * D;  // bytes of a tile's 64-dim half
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 8; ++r)
        put4(tile, half, row0 % 128 + g + 8 * i, r, pr, E[r][0][2 * i], E[r][0][2 * i + 1], E[r][1][2 * i], E[r][1][2 * i + 1]);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the kernel before this one has ended when this one has)
}

// ---------------------------------------------------------------------------
// Softmax groups
// ---------------------------------------------------------------------------
// The running max moved after c chunks of a tile: O (unless the tile is the item's first) and the
// tile's weights so far are scaled by f.
__device__ __forceinline__ void move_max(uint32_t s_col, uint32_t o_col, int c, bool have_o, float f) {
  if (have_o) {
#pragma unroll 1
    for (int x = 0; x < 8; ++x) {
      uint32_t o[16];
      tm_ld16(o_col + 16u * x, o);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
      tm_st16(o_col + 16u * x, o);
    }
  }
  const __half2 f2 = __float2half2_rn(f);
#pragma unroll 1
  for (int x = 0; x < c; ++x) {
    uint32_t w[16];
    tm_wait_st();
    tm_ld16(s_col + 16u * x, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = as_u32(__hmul2(as_h2(w[i]), f2));
    tm_st16(s_col + 16u * x, w);
  }
}

__device__ __forceinline__ bool softmax_role(const PfArgs& a, PfSmem& sm, Cursor cur, int warp, int lane, uint32_t& copies) {
  const int group = warp >> 2, wq = warp & 3;
  const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
  const uint32_t s_col = sm.tmem + 128u * group + lane_base, o_col = sm.tmem + 256u + 128u * group + lane_base;
  Piece p;
  uint32_t tiles = 0;       // of this group, over all pieces
  copies = 0;               // query operands copied
  int tg0 = 0;              // tiles of the CTA before this piece
  while (next_piece(a, cur, p)) {
    const int first = p.dual ? group : 0;
    const bool some = first < p.m;  // else nothing here waits for the MMAs, and no barrier may move
    if (some && wq == 0 && lane == 0) {
      // (the group's MMAs that read the previous operand have finished: pv_done was waited for)
      const RowSet& r = p.own ? a.ro : a.rp;
      const unsigned char* src = q_tile(a, p.own, p.item, p.dual ? 0 : group);
      const int rows = p.dual ? p.rows : min(128, p.rows - 128 * group);
      const uint32_t bytes = (uint32_t)((rows + 7) / 8 * 8) * 128u, dst = sm_addr(sm.q[group]), bar = sm_addr(&sm.q_full[group]);
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(2u * bytes) : "memory");
      bulk_g2s(dst, src, bytes, bar);
      bulk_g2s(dst + PF_HALF, src + (int64_t)r.hr * D, bytes, bar);
      ++copies;
    }
    const int row = (p.dual ? 0 : 128 * group) + 32 * wq + lane;  // within the 256-row tile
    const bool warp_live = (p.dual ? 0 : 128 * group) + 32 * wq < p.rows;
    const int c_of_row = p.own ? (256 * p.rt + row) / a.G : 0;
    float m = NEG_BIG, l = 0.f;
    for (int t = first; t < p.m; t += p.dual ? 2 : 1, ++tiles) {
      if (!bar_wait(&sm.s_full[group], tiles, &sm.fail)) return false;
      if (warp_live) {
        tc_after();
        const PfInfo info = sm.info[(tg0 + t) & 3];
        const int limit = min(info.nvalid, info.base + info.step * c_of_row);
        const bool masked = __any_sync(0xffffffffu, limit < BLK);
        float lt = 0.f;
        // the weights of columns 32 c .. + 31, whose scores s holds
        const auto chunk = [&](const int c, uint32_t (&s)[32]) {
          if (masked) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i >= limit) s[i] = 0xFF800000u;  // -inf
          }
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[i]);
#pragma unroll
          for (int i = 4; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
          const float top = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), info.ka, info.lv);
          if (__any_sync(0xffffffffu, top > m + PF_SLACK)) {
            const float mn = fmaxf(m, top), f = ex2(m - mn);
            m = mn;
            l *= f;
            lt *= f;
            move_max(s_col, o_col, c, t != first, f);
          }
          const float off = info.lv - m;
          const uint64_t ka2 = pack_f2(info.ka, info.ka), off2 = pack_f2(off, off);
          uint64_t sum[2] = {0ull, 0ull};
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float e0, e1;
            unpack_f2(fma_f2(pack_f2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), ka2, off2), e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            sum[i & 1] = add_f2(sum[i & 1], pack_f2(e0, e1));
            w[i] = pack_h2(e0, e1);
          }
          float a0, a1;
          unpack_f2(add_f2(sum[0], sum[1]), a0, a1);
          lt += a0 + a1;
          tm_st16(s_col + 16u * c, w);
        };
        // each chunk's columns are requested before the previous one is worked on; the
        // weights of chunk c overwrite columns 16 c .. + 15, which have been read by then
        uint32_t sa[32], sb[32];
        tm_ld32_async(s_col, sa);
#pragma unroll 1
        for (int c = 0; c < 4; c += 2) {  // (rolled: half the instructions to fetch)
          tm_ready32(sa);
          tm_ld32_async(s_col + 32u * c + 32u, sb);
          chunk(c, sa);
          tm_ready32(sb);
          if (c == 0) tm_ld32_async(s_col + 64u, sa);
          chunk(c + 1, sb);
        }
        l = fmaf(lt, info.iva, l);
        if (limit > info.vbad) l = __int_as_float(0x7fc00000);  // a value it sees is not finite
        tm_wait_st();
        tc_before();
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&sm.p_full[group]);
    }
    // ---- this group's partial of the item ----
    const int hr = p.own ? a.ro.hr : a.rp.hr;
    const int64_t row0 = slot_row(a, p.own, p.item, blockIdx.x);
    const int srow = (p.dual ? group * hr : 128 * group) + 32 * wq + lane;
    if (some && !bar_wait(&sm.pv_done[group], tiles - 1u, &sm.fail)) return false;
    if (warp_live) {
      tc_after();
      if (row < p.rows) a.ml[row0 + srow] = make_float2(m, l);
      if (some) {
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          uint32_t o[32];
          tm_ld32(o_col + 32u * x, o);
          if (row < p.rows) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(a.acc + acc_off(row0, hr, srow, 32 * x + i)) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
      }
      tc_before();
    }
    if (warp == 0 && lane == 0) {
      int2* e = a.tab + (p.own ? (int64_t)a.H * a.rp.rt : 0) + p.item;
      if (p.j == 0) e->x = blockIdx.x;
      if (p.j + p.m == p.s.tiles) e->y = blockIdx.x;
    }
    tg0 += p.m;
  }
  return true;
}

template <int MK, int MV, bool DQ>
__global__ void __launch_bounds__(PF_THREADS, 1) prefix_kernel(const __grid_constant__ PfArgs a) {
  extern __shared__ unsigned char smem_raw[];
  PfSmem& sm = *reinterpret_cast<PfSmem*>(smem_raw + ((1024u - (sm_addr(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- this CTA's range of the tiles ----
  const int nseg = a.H + (a.ro.rows > 0 ? a.B * a.H : 0);  // (own parts only where they are tiles)
  const int per = (nseg + PF_THREADS - 1) / PF_THREADS;
  long long sum = 0;
  bool short_window = false;
  for (int s = tid * per; s < min(nseg, (tid + 1) * per); ++s) {
    const Seg g = seg_info(a, s);
    sum += (long long)seg_units(g) * (s >= a.H ? a.ro.rt : a.rp.rt);
    short_window |= s >= a.H && a.causal && a.C > 1 && g.nw < a.C;
  }
  if (short_window && blockIdx.x == 0 && a.status) atomicOr(a.status, 8);
  long long inc = sum;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, x);
    if (lane >= x) inc += y;
  }
  if (lane == 31) sm.scan[warp] = inc;
  // codebooks while the counters arrive
  for (int i = tid; i < 2 * NCODES; i += PF_THREADS) {
    float c[SUB];
    const int code = i & (NCODES - 1);
    load8<NSN_DTYPE_F32>(i < NCODES ? a.cbk : a.cbv, (int64_t)code * SUB, c);
    const uint4 row = pack8_f16(c);
    uint4* dst = i < NCODES ? &sm.cbk[code][0] : &sm.cbv[code][0];
#pragma unroll
    for (int r = 0; r < 8; ++r) dst[(r + code) & 7] = row;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&sm.q_full[i], 1);
      bar_init(&sm.s_full[i], 1);
      bar_init(&sm.p_full[i], 4);
      bar_init(&sm.pv_done[i], 1);
    }
    for (int i = 0; i < PF_RING; ++i) {
      bar_init(&sm.full[i], PF_DEQ_WARPS);
      bar_init(&sm.empty[i], 2);
    }
    bar_init(&sm.meet, PF_DEQ_WARPS);
    bar_init(&sm.drain, 1);
    sm.fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < PF_THREADS / 32; ++w) {
    if (w < warp) before += sm.scan[w];
    total += sm.scan[w];
  }
  // at least one unit each, so the CTAs with tiles of an item are consecutive
  // (nothing above depends on the kernel before this one in the stream; the join, which does, may
  // be scheduled from here on and waits for this kernel's end)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const long long ctas = min((long long)gridDim.x, total), bid = blockIdx.x;
  if (bid >= ctas) return;  // the whole CTA: nothing to do
  const long long begin = total * bid / ctas, end = total * (bid + 1) / ctas;
  long long at = before + inc - sum;  // tiles before this thread's segments
  if (at <= begin && begin < at + sum) {
    for (int s = tid * per;; ++s) {
      const int units = seg_units(seg_info(a, s));
      const long long here = (long long)units * (s >= a.H ? a.ro.rt : a.rp.rt);
      if (begin < at + here) {
        sm.seg0 = s;
        sm.rt0 = (int)((begin - at) / units);
        sm.u0 = (int)((begin - at) % units);
        sm.units = end - begin;
        break;
      }
      at += here;
    }
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sm_addr(&sm.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();

  Cursor cur = {sm.seg0, sm.rt0, sm.u0, sm.units};
  bool ok = true;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PF_REGS_SOFTMAX));
    uint32_t copies;
    ok = softmax_role(a, sm, cur, warp, lane, copies);
    if (!ok && copies > 0) {  // a copy in flight lands before the CTA ends
      int never = 0;
      bar_wait(&sm.q_full[warp >> 2], copies - 1u, &never);
    }
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PF_REGS_DECODE));
    ok = decode_role<MK, MV, DQ>(a, sm, cur, warp - 8, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PF_REGS_MMA));
    if (warp == 16) {
      ok = mma_role(a, sm, cur);
      if (!ok) {  // let MMAs in flight finish before tensor memory is given back
        int never = 0;
        tc_commit_to(&sm.drain);
        bar_wait(&sm.drain, 0u, &never);
      }
    }
  }
  if (!ok) {
    *(volatile int*)&sm.fail = 1;
    if (a.status) atomicOr(a.status, 2);
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sm.tmem));
}

// ---------------------------------------------------------------------------
// Join: WPR warps per output row.  The partials of the row's prefix item and of its own part are
// weighted by 2^(m - max); the sum goes back through H and is rounded to the output type.
// ---------------------------------------------------------------------------
constexpr int JOIN_WARPS = 4;
constexpr int JOIN_DEPTH = 8;  // partials read at once

// Partials wi, wi + WPR, ... of one item, added to (m, l, v).
template <int WPR>
__device__ __forceinline__ void join_item(const PfArgs& a, bool own, int seg, int row, int wi, int lane, float& m, float& l, float (&v)[4]) {
  const RowSet& r = own ? a.ro : a.rp;
  const int64_t item = (int64_t)(own ? seg - a.H : seg) * r.rt + row / 256;
  const int tiles = seg_info(a, seg).tiles;
  const int2 ctas = a.tab[(own ? (int64_t)a.H * a.rp.rt : 0) + item];
  if (tiles == 0) return;  // (then the table says nothing)
  const int in = row % 256;
  const bool dual = min(256, r.rows - 256 * (row / 256)) <= 128;
  const int n = (((ctas.y - ctas.x + 1) << (dual ? 1 : 0)) - wi + WPR - 1) / WPR;  // of this warp
  // partial e: rows `in` (and, of alternating groups, hr + in) of the item's e-th slot
  const int64_t row0 = slot_row(a, own, item, ctas.x);
  const auto at = [&](int x) { const int e = x * WPR + wi; return dual ? row0 + (int64_t)(e >> 1) * 2 * r.hr : row0 + (int64_t)e * 2 * r.hr; };
  const auto srow = [&](int x) { const int e = x * WPR + wi; return dual && (e & 1) ? in + r.hr : in; };
  for (int e0 = 0; e0 < n; e0 += 32) {
    float2 mine = make_float2(NEG_BIG, 0.f);
    if (e0 + lane < n) mine = a.ml[at(e0 + lane) + srow(e0 + lane)];
    const bool some = mine.y != 0.f;  // (NaN counts)
    const unsigned have = __ballot_sync(0xffffffffu, some);
    const int cnt = min(32, n - e0);
    float mn = m, w = 0.f;
#pragma unroll 1
    for (int x0 = 0; x0 < cnt; x0 += JOIN_DEPTH) {
      float4 y[JOIN_DEPTH];
#pragma unroll
      for (int x = 0; x < JOIN_DEPTH; ++x) {
        y[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int e = x0 + x;
        if (e < 32 && (have >> e & 1u))
          y[x] = *reinterpret_cast<const float4*>(a.acc + acc_off(at(e0 + e), r.hr, srow(e0 + e), 4 * lane));
      }
      if (x0 == 0) {  // the weights, while the first sums are on their way
        mn = fmaxf(m, warp_max(some ? mine.x : NEG_BIG));
        const float f = ex2(m - mn);
        w = some ? ex2(mine.x - mn) : 0.f;
        l = l * f + warp_sum(some ? w * mine.y : 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= f;
        m = mn;
      }
#pragma unroll
      for (int x = 0; x < JOIN_DEPTH; ++x) {
        const float wx = __shfl_sync(0xffffffffu, w, (x0 + x) & 31);
        v[0] = fmaf(wx, y[x].x, v[0]);
        v[1] = fmaf(wx, y[x].y, v[1]);
        v[2] = fmaf(wx, y[x].z, v[2]);
        v[3] = fmaf(wx, y[x].w, v[3]);
      }
    }
  }
}

template <int WPR>
__global__ void __launch_bounds__(32 * JOIN_WARPS) prefix_join_kernel(const __grid_constant__ PfArgs a, void* __restrict__ out, int odt) {
  __shared__ float4 sv[JOIN_WARPS][32];
  __shared__ float2 sml[JOIN_WARPS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wi = warp % WPR;
  const int64_t r = ((int64_t)blockIdx.x * JOIN_WARPS + warp) / WPR;  // (b, c, head)
  const int nh = a.H * a.G;
  const bool live = r < (int64_t)a.B * a.C * nh;
  float2 own = make_float2(NEG_BIG, 0.f);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = NEG_BIG, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    if (a.own_lse && wi == 0) {
      own = a.own_lse[r];
      o = *reinterpret_cast<const float4*>(a.own_out + r * D + 4 * lane);
    }
    const int hq = (int)(r % nh), bc = (int)(r / nh), c = bc % a.C, b = bc / a.C, h = hq / a.G, gi = hq % a.G;
    join_item<WPR>(a, false, h, (b * a.C + c) * a.G + gi, wi, lane, m, l, v);
    if (!a.own_lse) join_item<WPR>(a, true, a.H + b * a.H + h, c * a.G + gi, wi, lane, m, l, v);
  }
  if constexpr (WPR > 1) {  // the row's first warp adds the others' sums
    sv[warp][lane] = make_float4(v[0], v[1], v[2], v[3]);
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (wi > 0) return;
#pragma unroll
    for (int x = 1; x < WPR; ++x) {
      const float2 ml = sml[warp + x];
      const float4 y = sv[warp + x][lane];
      if (ml.y == 0.f) continue;
      const float mn = fmaxf(m, ml.x), f = ex2(m - mn), w = ex2(ml.x - mn);
      l = l * f + ml.y * w;
      v[0] = v[0] * f + y.x * w;
      v[1] = v[1] * f + y.y * w;
      v[2] = v[2] * f + y.z * w;
      v[3] = v[3] * f + y.w * w;
      m = mn;
    }
  }
  if (!live) return;
  fwht128_warp(v, lane);
  // the own rows are in the original domain and divided by their denominator already
  const float mn = fmaxf(m, own.y != 0.f ? own.x : NEG_BIG);
  const float fr = l != 0.f ? ex2(m - mn) : 0.f, fo = own.y != 0.f ? ex2(own.x - mn) * own.y : 0.f;
  const float den = l * fr + fo;
  const float inv = den != 0.f ? 1.f / den : 0.f;  // no token at all: zeros
  const float ov[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (v[i] * (PF_INV_SQRT_D * fr) + ov[i] * fo) * inv;
  const int64_t off = r * D + 4 * lane;
  if (odt == NSN_DTYPE_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + off) = make_float4(v[0], v[1], v[2], v[3]);
  } else if (odt == NSN_DTYPE_BF16) {
    __nv_bfloat162 x[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + off) = *reinterpret_cast<const uint2*>(x);
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + off) = make_uint2(pack_h2(v[0], v[1]), pack_h2(v[2], v[3]));
  }
}

RowSet row_set(int64_t rows) {
  RowSet r;
  r.rows = (int)rows;
  r.rt = (int)((rows + 255) / 256);
  r.hr = rows > 128 ? 128 : (int)((rows + 31) / 32 * 32);
  return r;
}

// With one query per sequence the own part has 1 to 8 rows per (b, kv-head): too few for a
// 128-row tile, and the decode kernel takes it.  Longer chunks take tiles for both parts.
bool own_by_decode(int n_queries) { return n_queries == 1; }

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: (own part by decode: its workspace, whose counters come first, then its rows and their
// denominators), the query tiles, the item table, the (m, l) pairs and the sums of every slot.
struct PfLayout {
  RowSet rp, ro;
  size_t own_out, own_lse, qt, tab, ml, acc, bytes;
};
PfLayout layout(int B, int H, int g, int C, int own_capacity) {
  PfLayout y;
  const bool dec = own_by_decode(C);
  y.rp = row_set((int64_t)B * C * g);
  y.ro = row_set(dec ? 0 : (int64_t)C * g);
  const int64_t ip = (int64_t)H * y.rp.rt, io = (int64_t)B * H * y.ro.rt, rows_out = (int64_t)B * C * H * g;
  const int64_t rows = (ip + PF_CTAS) * 2 * y.rp.hr + (io + PF_CTAS) * 2 * y.ro.hr;
  // (the counters' place is kept for any C, so that one zero-filled workspace serves calls of several)
  y.own_out = up256(dec ? decode_workspace_bytes(B, H, decode_geometry(B, own_capacity, H * g, H)) : decode_counter_bytes(B, H));
  y.own_lse = y.own_out + (dec ? up256((size_t)rows_out * D * sizeof(float)) : 0);
  y.qt = y.own_lse + (dec ? up256((size_t)rows_out * sizeof(float2)) : 0);
  y.tab = y.qt + up256((size_t)(ip * 2 * q_tile_bytes(y.rp) + io * 2 * q_tile_bytes(y.ro)));
  y.ml = y.tab + up256((size_t)(ip + io) * sizeof(int2));
  y.acc = y.ml + up256((size_t)rows * sizeof(float2));
  y.bytes = y.acc + (size_t)rows * D * sizeof(float);
  return y;
}

// A launch that may be scheduled before the kernel in front of it in the stream has ended; the
// kernel waits (griddepcontrol.wait) before it reads what that one wrote.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, bool early, cudaStream_t s, A... args) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <int MK, int MV, bool DQ>
cudaError_t launch_t(const PfArgs& a, int ctas, cudaStream_t s) {
  const size_t smem = sizeof(PfSmem) + 1024;
  const cudaError_t e = cudaFuncSetAttribute(prefix_kernel<MK, MV, DQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_early(prefix_kernel<MK, MV, DQ>, ctas, PF_THREADS, smem, true, s, a);
}

}  // namespace

size_t prefix_workspace_bytes(int batch, int n_kv_heads, int g, int n_queries, int own_capacity) {
  return layout(batch, n_kv_heads, g, n_queries, own_capacity).bytes;
}

cudaError_t launch_prefix(const CacheView& pk, const CacheView& pv, const CacheView& k, const CacheView& v, const void* q,
                          int dtype, int n_q_heads, int n_queries, bool causal, int64_t qsb, int64_t qst, int64_t qsh,
                          float softmax_scale, const float* cbk, const float* cbv, void* out, int out_dtype, void* ws,
                          cudaStream_t s) {
  PfArgs a;
  a.pk = pk; a.pv = pv; a.k = k; a.v = v;
  a.q = q;
  a.dtype = dtype;
  a.qsb = qsb; a.qst = qst; a.qsh = qsh;
  a.qscale = softmax_scale * PF_LOG2E * PF_INV_SQRT_D;
  a.cbk = cbk; a.cbv = cbv;
  a.B = k.batch; a.C = n_queries; a.H = k.n_kv_heads; a.G = n_q_heads / k.n_kv_heads;
  a.causal = causal ? 1 : 0;
  const PfLayout y = layout(a.B, a.H, a.G, a.C, k.capacity);
  a.rp = y.rp;
  a.ro = y.ro;
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.qt = w + y.qt;
  a.tab = reinterpret_cast<int2*>(w + y.tab);
  a.ml = reinterpret_cast<float2*>(w + y.ml);
  a.acc = reinterpret_cast<float*>(w + y.acc);
  a.own_out = nullptr;
  a.own_lse = nullptr;
  a.status = k.status;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int ctas = sms < PF_CTAS ? sms : PF_CTAS;
  if (own_by_decode(n_queries)) {
    float* oo = reinterpret_cast<float*>(w + y.own_out);
    float2* ol = reinterpret_cast<float2*>(w + y.own_lse);
    a.own_out = oo;
    a.own_lse = ol;
    e = launch_decode_lse(k, v, q, dtype, n_q_heads, qsb, qsh, softmax_scale, cbk, cbv, oo, ol, w,
                          decode_geometry(a.B, k.capacity, n_q_heads, a.H), s);
    if (e != cudaSuccess) return e;
  }
  const int64_t groups = (int64_t)a.H * ((a.rp.rows + 15) / 16) + (int64_t)a.B * a.H * ((a.ro.rows + 15) / 16);
  e = launch_early(prefix_query_kernel, (unsigned)((groups + QUERY_WARPS - 1) / QUERY_WARPS), 32 * QUERY_WARPS, 0,
                   a.own_lse != nullptr, s, a);
  if (e != cudaSuccess) return e;
  const bool k2 = k.mode == NSN_MODE_2BIT, v2 = v.mode == NSN_MODE_2BIT;
  if (k.dq)
    e = k2 ? (v2 ? launch_t<2, 2, true>(a, ctas, s) : launch_t<2, 1, true>(a, ctas, s))
           : (v2 ? launch_t<1, 2, true>(a, ctas, s) : launch_t<1, 1, true>(a, ctas, s));
  else
    e = k2 ? (v2 ? launch_t<2, 2, false>(a, ctas, s) : launch_t<2, 1, false>(a, ctas, s))
           : (v2 ? launch_t<1, 2, false>(a, ctas, s) : launch_t<1, 1, false>(a, ctas, s));
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.B * a.C * n_q_heads;
  // few rows: four warps each, so that the partials are read in one or two rounds
  if (rows <= (int64_t)PF_CTAS * 16)
    return launch_early(prefix_join_kernel<JOIN_WARPS>, (unsigned)rows, 32 * JOIN_WARPS, 0, true, s, a, out, out_dtype);
  return launch_early(prefix_join_kernel<1>, (unsigned)((rows + JOIN_WARPS - 1) / JOIN_WARPS), 32 * JOIN_WARPS, 0, true, s, a,
                      out, out_dtype);
}

}  // namespace nsn

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
// One CTA: 20 warps, two of them idle (registers move between whole warpgroups).
//   warps 8-11, 12-15  decode K tiles and V tiles into shared memory: a lane takes one token, gathers
//               its codewords (4-fold replicated fp16 codebook), applies signs, scale and mean in
//               fp16, and stores 16-byte chunks of the 128-byte-swizzled operand tile;
//   warps 16, 17  issue the MMAs of one softmax group each: S = Q K^T (both from shared memory) into tensor
//               memory and O += P V (P from tensor memory);
//   warps 0-3, 4-7  two softmax groups, each with its own S/P and O columns: a thread owns one
//               query row, so the softmax needs no exchange between lanes.
// With more than 128 rows in an item's tile the groups take 128 rows each and share every K/V
// tile; otherwise both take the same rows and alternate token tiles, as two partials.
//
// Scales: inside a block the fp16 rows are y_t / smax (smax = the largest s1 of the block), so
// they are of order one whatever the norms are; smax of K multiplies the scores, log2 smax of
// V goes into the exponent (so w is scaled by what it contributes, not by what it weighs) and
// its inverse into the denominator.  (A window tile's scale: window_scale.)  Rounding to fp16
// happens at q~, y and w (2^-11 relative at most each; y has three: its scale, its mean's product,
// its sum): the operands of the tensor cores, which in 32 bits would neither fit in shared memory
// nor reach this rate.  Sums, maxima and the denominator are fp32.
//
// What bounds it.  Per 128 tokens and 256 rows the products take 2048 tensor cycles, the
// exponentials 2048, the operands and the decoding about 3900 of shared memory.  Measured (2-bit,
// 8 kv-heads): 256 rows per kv-head over 131072 tokens 168 us, 54 % of the cycles in the tensor
// cores; 4096 rows over 32768 tokens 572 us, 0.96 PFLOP/s; 64 rows over 32768 tokens 51 us.  A tile
// takes about 4700 cycles: the decode teams' instructions (one warp of each per scheduler, some 600 a
// tile) and the softmax share the issue slots.  What brought it there, at 4096 rows: two decode teams, half tiles in flight and an
// MMA warp per group 745 -> 609 us, codeword reads ahead of writes 609 -> 573; V's scales left by the V
// team, at 64 rows 55 -> 51.  Not kept: one buffer
// of half tiles instead of two whole ones, with room for 8 replicas (668), three buffers with one
// decode team (745), softmax turns between the groups (no change).

#include "hadamard_mma.cuh"
#include "nsn_launch.h"

namespace nsn {
namespace {

constexpr float PF_LOG2E = 1.4426950408889634f;
constexpr float PF_INV_SQRT_D = 0.08838834764831845f;  // 1/sqrt(128)
constexpr int PF_CTAS = 148;       // at most; one per SM
constexpr int PF_DEQ_WARPS = 8;    // two teams, one for K tiles and one for V tiles
constexpr int PF_TEAM = 4;
constexpr int PF_THREADS = 32 * (8 + PF_DEQ_WARPS + 4);  // the last warpgroup: the MMA warps and two idle ones
// Registers per thread after the roles part: at launch all 20 warps hold 96, so the sum over
// the warps may not pass 20 x 96 = 1920: 8 x 104 + 8 x 120 + 4 x 32.
constexpr int PF_REGS_SOFTMAX = 104, PF_REGS_DECODE = 120, PF_REGS_MMA = 32;
static_assert(8 * PF_REGS_SOFTMAX + PF_DEQ_WARPS * PF_REGS_DECODE + 4 * PF_REGS_MMA <= (PF_THREADS / 32) * 96, "registers of the CTA");
constexpr int PF_BUFS = 2;         // buffers of K tiles, and of V tiles, in shared memory (tile g of the CTA in buffer g & 1)
constexpr int PF_REP = 4;          // replicas of each codeword
constexpr int PF_TILE_BYTES = 32768;  // 128 tokens (or rows) x 128 dims fp16: two 16 KB halves of 64 dims
constexpr uint32_t PF_HALF = 16384u;
// The reference m_i of a row's weights is set PF_HEAD below its largest score, and moves only when a score
// exceeds it by more than PF_HEAD + PF_SLACK (log2 units): most tiles leave O alone, and weights stay below 2^15
// (fp16 ends at 65504).  fp16 steps by 2^-24 at the low end, so a weight is off by at most 2^-32 of the row's
// largest (or by its rounding), which counts where one token has nearly all the weight and thousands share the
// rest: with m_i at the largest score, 14k tokens 17.7 nats below a first token lost most of what they weigh
// (0.2-0.4 % of the output, with its value a twentieth of theirs; now under 0.06 %, the rounding of its row).
constexpr float PF_HEAD = 7.0f, PF_SLACK = 8.0f;
// The scale of a V tile without a value other than zero (a power of two below every fp16 norm): it adds nothing
// to the sum, so its scores must not raise the reference of rows that weigh small values; its weights still count
// in the denominator.
constexpr float PF_ZERO_V = 9.094947017729282e-13f;  // 2^-40
constexpr uint32_t PF_WAIT_LIMIT = 1u << 22;   // attempts of a wait before it gives up (seconds)
constexpr uint32_t PF_POLL_LIMIT = 1u << 26;   // idle rounds of an MMA warp's event loop (seconds)

struct RowSet {  // the rows of one kind of segment
  int rows;      // query rows of a segment
  int rt;        // 256-row tiles
  int hr;        // rows of one group's half of a partial slot (128, or the rows rounded up to 32)
  int cost;      // of an item beside its tiles, in tiles
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
  int32_t* bad;            // a CTA gave up: the join writes NaN (and reads neither the table nor partials)
  int give_up;             // the CTA whose K team gives up at once (-1: none), for the diagnostic of this path
  float2* ml;              // partial (m, l): prefix slots, then own slots
  float* acc;              // partial sums, same slots
  const float* own_out;    // not null: the own part's rows come from the decode kernel (then ro is empty),
  const float2* own_lse;   //   each with its (max in log2 units, denominator)
  int32_t* status;
};

struct PfInfo {            // of one K tile, for the softmax
  float ka;                // scale
  int nvalid;              // tokens
  int base, step;          // a query at chunk position c sees base + step c of them (window tile of a causal segment)
};
struct PfInfoV {           // of one V tile
  float lv, iva;           // log2 and inverse of its scale
  int vbad;                // first token whose row is not finite (128: none)
  int pad;
};

struct PfSmem {
  alignas(1024) unsigned char q[2][PF_TILE_BYTES];
  alignas(1024) unsigned char kv[2][PF_BUFS][PF_TILE_BYTES];  // K tiles, V tiles
  alignas(128) uint4 cbk[NCODES][PF_REP];
  alignas(128) uint4 cbv[NCODES][PF_REP];
  alignas(16) unsigned char o[PF_DEQ_WARPS][256];  // the mean row of the tile a decode warp is at
  alignas(16) PfInfo info[4];
  alignas(16) PfInfoV info_v[4];
  float red[2][2][PF_TEAM], red_base[2][2][PF_TEAM];  // per team (double-buffered: window tiles in turn): the tile's scale
  int red_bad[2][2][PF_TEAM];
  alignas(8) uint64_t q_full[2], s_full[2][2], p_full[2][2], pv_done[2][2], full[2][PF_BUFS], empty[2][PF_BUFS], meet[2], v_info[4], drain[2];
  long long scan[PF_THREADS / 32];
  long long units;
  int seg0, rt0, u0;
  uint32_t tmem;
  int fail;
};
static_assert(sizeof(PfSmem) <= 232448, "shared memory of one SM");

// ---------------------------------------------------------------------------
// Barriers, tensor core and tensor memory
// ---------------------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_addr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_addr(b)) : "memory");
}
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done) : "r"(smem_addr(b)), "r"(parity & 1u) : "memory");
  return done != 0;
}
// Bounded wait; false if it gave up or another role did.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, volatile int* fail) {
  for (uint32_t i = 0; i < PF_WAIT_LIMIT; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(smem_addr(b)), "r"(parity & 1u) : "memory");
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
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_addr(b)) : "memory");
}

// Matrix descriptors of the 128-byte-swizzled operands (descriptor version 1, layout 2): 8-row
// groups of 128-byte rows 1024 B apart; the leading offset is the distance of the two 64-dim
// halves where the operand is read across them (V: dims are the N axis).
// kind::f16, fp32 accumulator, fp16 operands, M = 128; S: N = 64 tokens; O: N = 128 dims, V read with
// its N axis (dims) contiguous.
constexpr uint32_t PF_IDESC_QK = (1u << 4) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t PF_IDESC_PV = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

// The K = 16 steps of one product, issued by one elected lane of a converged warp: with operands uniform
// across the warp the compiler keeps them in uniform registers.  From a single-lane branch, where each
// operand is moved there first, an MMA took over 100 cycles to issue beside the busy warps, twice its
// execution.  A descriptor is its low word (start address and leading
// offset) and the constant high word.
constexpr uint32_t PF_DESC_HI = (uint32_t)(((1024ull >> 4 << 32) | (1ull << 46) | (2ull << 61)) >> 32);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }
// S = Q K^T: 32 bytes of dims a step within the 128-byte rows, then the other 64-dim half (16 KB on).
__device__ __forceinline__ void mma_qk(uint32_t d, uint32_t a, uint32_t b) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 da, db;\n .reg .b32 x, y;\n elect.sync _|e, 0xffffffff;\n"
      " add.u32 x, %1, 0;\n add.u32 y, %2, 0;\n mov.b64 da, {x, %4};\n mov.b64 db, {y, %4};\n"
      " setp.ne.b32 p, 0, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n"
      " add.u32 x, %1, 2;\n add.u32 y, %2, 2;\n mov.b64 da, {x, %4};\n mov.b64 db, {y, %4};\n"
      " setp.eq.b32 p, 0, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n"
      " add.u32 x, %1, 4;\n add.u32 y, %2, 4;\n mov.b64 da, {x, %4};\n mov.b64 db, {y, %4};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n"
      " add.u32 x, %1, 6;\n add.u32 y, %2, 6;\n mov.b64 da, {x, %4};\n mov.b64 db, {y, %4};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n"
      " add.u32 x, %1, 1024;\n add.u32 y, %2, 1024;\n mov.b64 da, {x, %4};\n mov.b64 db, {y, %4};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n"
      " add.u32 x, %1, 1026;\n add.u32 y, %2, 1026;\n mov.b64 da, {x, %4};\n mov.b64 db, {y, %4};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n"
      " add.u32 x, %1, 1028;\n add.u32 y, %2, 1028;\n mov.b64 da, {x, %4};\n mov.b64 db, {y, %4};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n"
      " add.u32 x, %1, 1030;\n add.u32 y, %2, 1030;\n mov.b64 da, {x, %4};\n mov.b64 db, {y, %4};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n"
      "}\n"
      ::"r"(d), "r"(a), "r"(b), "r"(PF_IDESC_QK), "r"(PF_DESC_HI) : "memory");
}
// O (+)= P V over 64 tokens: 8 columns of P and 16 token rows (2 KB) of V a step.
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 db;\n .reg .b32 x, y;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " add.u32 x, %1, 0;\n add.u32 y, %2, 0;\n mov.b64 db, {y, %5};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n"
      " add.u32 x, %1, 8;\n add.u32 y, %2, 128;\n mov.b64 db, {y, %5};\n"
      " setp.eq.b32 p, 0, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n"
      " add.u32 x, %1, 16;\n add.u32 y, %2, 256;\n mov.b64 db, {y, %5};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n"
      " add.u32 x, %1, 24;\n add.u32 y, %2, 384;\n mov.b64 db, {y, %5};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n"
      "}\n"
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
__device__ __forceinline__ void tm_ready64(uint32_t (&r)[32], uint32_t (&q)[32]) {
  tm_ready32(r);
  tm_ready32(q);
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

__device__ __forceinline__ float minus_inf() { return __int_as_float(0xFF800000); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// A value that all lanes hold, in a form that the compiler knows to be warp-uniform (a reduction's
// result is): the MMA operands derived from it then stay in uniform registers.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

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
// Ranges are cut in units of one tile plus `cost` for each item (its query operand, the latency of its
// first scores and its partial, which are not overlapped with the same group's other items).
__device__ __forceinline__ int seg_units(const Seg& s, const RowSet& r) { return s.tiles > 0 ? s.tiles + r.cost : 0; }
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
    const int units = seg_units(p.s, r), n = (int)min((long long)(units - c.u), c.left);
    p.j = max(0, c.u - r.cost);
    p.m = max(0, c.u + n - r.cost) - p.j;
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
// What a lane reads for one K or V tile of a quantized block: token 32 w + lane of it (w: the warp
// within its team), and what the block's largest s1 needs.
struct Raw {
  uint4 code, sign;
  uint32_t norm, level;   // fp16 (s1, s2); or fp16 s2, and the byte with the s1 level
  uint4 four;             // s1 of tokens 4 lane .. 4 lane + 3 (fp16 pairs, or levels)
  uint2 mean;             // dims 4 lane .. + 3
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
    four.x = ld_u16(c.levels + blk * (BLK / 2) + 2 * lane);
    par = ld_v2(c.params + blk * 16);
  } else {
    four = ld_v4(c.norms + blk * (4 * BLK) + 16 * lane);
  }
}

template <int MODE, bool DQ>
__device__ __forceinline__ void raw_load(Raw& r, const Src& c, int64_t blk, int w, int lane) {
  const int t = 32 * w + lane;
  r.code = ld_v4(c.codes + blk * (BLK * NSUB) + NSUB * t);
  if constexpr (MODE == NSN_MODE_2BIT) r.sign = ld_v4(c.signs + blk * (BLK * NSUB) + NSUB * t);
  if constexpr (DQ) {
    r.norm = ld_u16(c.norms + blk * (2 * BLK) + 2 * t);
    r.level = ld_u8(c.levels + blk * (BLK / 2) + t / 2);
    r.mean.x = ld_u16(c.means + blk * (D / 2) + 2 * lane);
  } else {
    r.norm = ld_u32(c.norms + blk * (4 * BLK) + 4 * t);
    r.mean = ld_v2(c.means + blk * (2 * D) + 8 * lane);
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

// Writes this warp's 32 rows of a decoded tile: fp16((u_hat s2 + o) s1 / smax) per token.
template <int MODE, bool DQ>
__device__ __forceinline__ void tile_write(const Raw& r, const uint4 (*cb)[PF_REP], unsigned char* tile, unsigned char* orow,
                                           float smax, int nvalid, int w, int lane) {
  const int row = 32 * w + lane;
  float s1, s2;
  uint2 mean = r.mean;
  if constexpr (DQ) {
    const float2 ls = lo_step(r.par.x), lo = lo_step(r.par.y);
    s1 = fmaf((float)((r.level >> (4 * (lane & 1))) & 15u), ls.y, ls.x);
    s2 = __low2float(as_h2(r.norm));
    const uint32_t v = r.mean.x;
    mean.x = pack_h2(fmaf((float)(v & 15u), lo.y, lo.x), fmaf((float)((v >> 4) & 15u), lo.y, lo.x));
    mean.y = pack_h2(fmaf((float)((v >> 8) & 15u), lo.y, lo.x), fmaf((float)(v >> 12), lo.y, lo.x));
  } else {
    const float2 n = __half22float2(as_h2(r.norm));
    s1 = n.x;
    s2 = n.y;
  }
  // Rows past the block's tokens come out as zeros: both scales 0, whatever their records hold.  A row that is not
  // finite comes out as NaN throughout, so that no score with it is minus infinity (0 x infinity is NaN; where smax
  // is 0, s1 is 0 or NaN).
  const bool live = row < nvalid;
  const __half2 zero2 = __float2half2_rn(0.f);
  const uint32_t odd = as_u32(__hfma2(as_h2(mean.x), zero2, __hmul2(as_h2(mean.y), zero2))) & 0x7FFF7FFFu;
  const float bad_mean = __any_sync(0xffffffffu, odd != 0u) ? __int_as_float(0x7fc00000) : 0.f;
  const float ratio = smax > 0.f ? s1 / smax : s1, scale = ratio * s2;
  const __half2 b2 = __float2half2_rn(live ? ratio + bad_mean : 0.f), a2 = __float2half2_rn(live ? fmaf(scale, 0.f, scale) : 0.f);
  __syncwarp();  // the previous tile's mean row has been read
  reinterpret_cast<uint2*>(orow)[lane] = mean;
  __syncwarp();
  unsigned char* dst = tile + row * 128;
  const uint4* rep = &cb[0][lane & (PF_REP - 1)];
  const uint32_t sw[4] = {r.sign.x, r.sign.y, r.sign.z, r.sign.w};
  // Four sub-vectors at a time, the next four's reads before this four's writes: the compiler keeps
  // reads behind writes that might alias them, and each would wait out the latency of the one before.
  uint4 c[2][4], o[2][4];
  const auto gather = [&](int s0, uint4 (&cw)[4], uint4 (&om)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // the record holds the even sub-vectors' codes, then the odd ones'
      const int s = s0 + i;
      const uint32_t word = (s & 1) ? ((s >> 1) < 4 ? r.code.z : r.code.w) : ((s >> 1) < 4 ? r.code.x : r.code.y);
      const uint32_t code = __byte_perm(word, 0u, 0x4440u | (uint32_t)((s >> 1) & 3));
      cw[i] = rep[code * PF_REP];
      om[i] = *reinterpret_cast<const uint4*>(orow + 16 * s);
    }
  };
  gather(0, c[0], o[0]);
#pragma unroll
  for (int s0 = 0; s0 < NSUB; s0 += 4) {
    const int now = (s0 >> 2) & 1;
    if (s0 + 4 < NSUB) gather(s0 + 4, c[now ^ 1], o[now ^ 1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = s0 + j;
      uint32_t u[4] = {c[now][j].x, c[now][j].y, c[now][j].z, c[now][j].w};
      const uint32_t om[4] = {o[now][j].x, o[now][j].y, o[now][j].z, o[now][j].w};
      if constexpr (MODE == NSN_MODE_2BIT) {  // the sign of dim 8 s + i is bit 15 - s of field i
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] ^= (sw[i] << s) & 0x80008000u;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = as_u32(__hfma2(as_h2(u[i]), a2, __hmul2(as_h2(om[i]), b2)));
      *reinterpret_cast<uint4*>(dst + (s >> 3) * PF_HALF + (((s & 7) ^ (row & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
}

// Window rows 16 w .. 16 w + 15 (w: a 16-row group) of one sequence as A fragments of the transform (rows past nw: zero).
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

// The largest mean square of those rows that are finite, that of the rows below `nbase`, and the first row that is
// not finite.
__device__ __forceinline__ void window_scan(const uint32_t (&f)[8][4], int w, int lane, int nbase, float& smax, float& sbase, int& bad) {
  smax = sbase = 0.f;
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
    const int row = 16 * w + (lane >> 2) + 8 * i;
    if (ss <= 3.0e38f) smax = fmaxf(smax, ss * (1.0f / D));
    else bad = min(bad, row);
    if (ss <= 3.0e38f && row < nbase) sbase = fmaxf(sbase, ss * (1.0f / D));
  }
  smax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(smax)));  // (neither is negative)
  sbase = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(sbase)));
  bad = __reduce_min_sync(0xffffffffu, bad);
}

// The scale of a window tile from those two mean squares: the power of two at or below the root of `sbase`, or 2^-11
// of the one for `smax` where that is larger (rows are then below 2^12 in the root mean square, elements below
// 46400; fp16 ends at 65504).  `sbase` is over the rows that every query of a chunk sees, so later tokens of the
// chunk change no bit of an earlier query unless they are over 2^11 times larger: a power of two scales exactly.
// From there on the scale follows them, and the other rows keep their precision until they are 2^-12 of it
// (an element is off by 2^-25 of the scale at most).  0: no row has a value other than zero.
__device__ __forceinline__ float window_scale(float smax, float sbase) {
  const int top = ((int)(__float_as_uint(smax) >> 23) - 127) >> 1, base = ((int)(__float_as_uint(sbase) >> 23) - 127) >> 1;
  return smax > 0.f ? __uint_as_float((uint32_t)(max(top - 11, base) + 127) << 23) : 0.f;
}

// Four consecutive dims 16 r + 4 p of row t of an operand tile, as fp16 (`half`: bytes between its 64-dim halves).
__device__ __forceinline__ void put4(unsigned char* tile, int64_t half, int t, int r, int p, float a, float b, float c, float d) {
  const int chunk = 2 * r + (p >> 1);
  unsigned char* dst = tile + (chunk >> 3) * half + t * 128 + (((chunk & 7) ^ (t & 7)) << 4) + (p & 1) * 8;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_h2(a, b), pack_h2(c, d));
}

// Writes those rows rotated, fp16(H x / smax); rows that are not finite are NaN throughout (no score with
// them is minus infinity), or zero where `drop` (V: a zero weight would not cancel them).
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
    const bool bad = !(fabsf(E[0][0][2 * i]) <= 3.0e38f);
    const float as = drop ? 0.f : __int_as_float(0x7fc00000);
#pragma unroll
    for (int r = 0; r < 8; ++r)
      put4(tile, PF_HALF, 16 * w + (lane >> 2) + 8 * i, r, lane & 3, bad ? as : E[r][0][2 * i] * inv, bad ? as : E[r][0][2 * i + 1] * inv,
           bad ? as : E[r][1][2 * i] * inv, bad ? as : E[r][1][2 * i + 1] * inv);
  }
}

// Meets the other warps of the team (bounded, as every wait here); `phase` counts the meetings.
__device__ __forceinline__ bool decode_sync(PfSmem& sm, int team, uint32_t& phase, int lane) {
  __syncwarp();
  if (lane == 0) bar_arrive(&sm.meet[team]);
  return bar_wait(&sm.meet[team], phase++, &sm.fail);
}

// One decode warp's walk over the pieces: the K team (TV = false) or the V team; the next tile's
// global reads are issued before the current one waits for its buffer.  Each team leaves its tiles'
// scales for the softmax: K's with the tile itself, V's, which the softmax needs before the tile, as
// soon as they are known (a slot's last reader was done before the team could get this far).
template <int MODE, bool DQ, bool TV>
__device__ __forceinline__ bool decode_role(const PfArgs& a, PfSmem& sm, Cursor cur, int w, int lane) {
  Piece p;
  int tg0 = 0;        // tiles of the CTA before this piece
  uint32_t met = 0;
  unsigned char* orow = sm.o[w + (TV ? PF_TEAM : 0)];
  const auto leave_v = [&](int g, float smax, int vbad) {
    if (w == 0 && lane == 0) {
      PfInfoV v;
      v.iva = smax > 0.f ? smax : PF_ZERO_V;
      v.lv = log2f(v.iva);
      v.iva = 1.f / v.iva;
      v.vbad = vbad;
      v.pad = 0;
      sm.info_v[g & 3] = v;
      bar_arrive(&sm.v_info[g & 3]);
    }
  };
  while (next_piece(a, cur, p)) {
    const CacheView& c = p.own ? (TV ? a.v : a.k) : (TV ? a.pv : a.pk);
    const int64_t seq = p.own ? p.seg - a.H : p.seg;
    const Src src = seq_src<DQ>(c, seq);
    Raw next, raw;
    const auto fetch = [&](int t) {
      if (p.j + t < p.s.blocks) raw_load<MODE, DQ>(next, src, p.j + t, w, lane);
    };
    fetch(0);
    for (int t = 0; t < p.m; ++t) {
      raw = next;
      if (t + 1 < p.m) fetch(t + 1);
      const int g = tg0 + t, buf = g & 1, blk = p.j + t;
      unsigned char* tile = sm.kv[TV][buf];
      PfInfo info;
      float smax;
      if (blk < p.s.blocks) {
        const int nvalid = min(BLK, p.s.nq - BLK * blk);
        smax = block_smax<DQ>(raw.four, raw.par, nvalid, lane);
        if constexpr (TV) leave_v(g, smax, BLK);
        if (g >= PF_BUFS && !bar_wait(&sm.empty[TV][buf], (uint32_t)(g / PF_BUFS - 1), &sm.fail)) return false;
        tile_write<MODE, DQ>(raw, TV ? sm.cbv : sm.cbk, tile, orow, smax, nvalid, w, lane);
        info.nvalid = info.base = nvalid;
        info.step = 0;
      } else {
        int vbad = BLK;
        uint32_t f[8][4];
        const uint32_t side = met & 1;
        const bool chunk = p.own && a.causal;
        const int nbase = chunk ? max(1, p.s.nw - a.C + 1) : p.s.nw;  // rows that every query sees (that sees any)
        float sbase = 0.f;
        smax = 0.f;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          float mine, base;
          int bad;
          window_load(f, c, seq, p.s.nw, 2 * w + i, lane);
          window_scan(f, 2 * w + i, lane, nbase, mine, base, bad);
          smax = fmaxf(smax, mine);
          sbase = fmaxf(sbase, base);
          vbad = min(vbad, bad);
        }
        if (lane == 0) {
          sm.red[TV][side][w] = smax;
          sm.red_base[TV][side][w] = sbase;
          sm.red_bad[TV][side][w] = vbad;
        }
        if (!decode_sync(sm, TV, met, lane)) return false;
#pragma unroll
        for (int x = 0; x < PF_TEAM; ++x) {
          smax = fmaxf(smax, sm.red[TV][side][x]);
          sbase = fmaxf(sbase, sm.red_base[TV][side][x]);
          vbad = min(vbad, sm.red_bad[TV][side][x]);
        }
        smax = window_scale(smax, sbase);
        if constexpr (TV) leave_v(g, smax, vbad);
        if (g >= PF_BUFS && !bar_wait(&sm.empty[TV][buf], (uint32_t)(g / PF_BUFS - 1), &sm.fail)) return false;
#pragma unroll 1
        for (int i = 1; i >= 0; --i) {  // (the second 16 rows are still in f)
          if (i == 0) window_load(f, c, seq, p.s.nw, 2 * w, lane);
          window_write(f, smax, TV, tile, 2 * w + i, lane);
        }
        info.nvalid = p.s.nw;
        info.step = chunk ? 1 : 0;
        info.base = info.step ? p.s.nw - a.C + 1 : p.s.nw;
      }
      if (!TV && w == 0 && lane == 0) {
        info.ka = smax > 0.f ? smax : 1.f;
        sm.info[g & 3] = info;
      }
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(&sm.full[TV][buf]);
    }
    tg0 += p.m;
  }
  return true;
}

// ---------------------------------------------------------------------------
// The MMA warps, one per softmax group (one warp for both spent longer issuing than the products
// took).  S and P of a group are two halves of 64 tokens: while the softmax works on one, the products
// of the other run, so its scores are there when it is done.  S = Q K^T of a half needs the K tile and
// its previous P consumed, O += P V the V tile and P.  Each warp walks every tile of every piece in
// order and frees it, by a commit behind its own products or, where the other group alone uses the
// tile, at once.  No tile is replaced before both warps have seen it, K tiles and V tiles have
// buffers and barriers of their own, each filled by one team in order: so whoever waits has seen the
// phase before the one it waits for, and a barrier's parity is never ambiguous.  The warps stay
// converged (votes decide).
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool test_all(uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, bar_test(b, parity)); }

__device__ __forceinline__ bool mma_role(const PfArgs& a, PfSmem& sm, Cursor cur, const int group) {
  constexpr uint32_t TILE = PF_TILE_BYTES >> 4;
  // descriptors differ from these only by constant steps of the start address (16-byte units)
  const uint32_t tmem = (uint32_t)uniform((int)sm.tmem);
  const uint32_t s_col = tmem + 128u * group, o_col = tmem + 256u + 128u * group;
  const uint32_t q_lo = desc_lo(smem_addr(sm.q[0]), 16u) + TILE * group, k_lo = desc_lo(smem_addr(sm.kv[0][0]), 16u),
                 v_lo = desc_lo(smem_addr(sm.kv[1][0]), PF_HALF);
  uint64_t *s_full = sm.s_full[group], *p_full = sm.p_full[group], *pv_done = sm.pv_done[group];
  Piece p;
  int g0 = 0, pieces = 0;                  // tiles and pieces before this piece
  int seen[2] = {0, 0};                    // K and V tiles seen, over all pieces
  uint32_t done = 0u, built = 0u;          // tiles finished and query operands used, over all pieces
  uint32_t idle = 0;
  while (next_piece(a, cur, p)) {
    const int m = uniform(p.m), step = uniform(p.dual ? 2 : 1), first = step == 2 ? (group + pieces) & 1 : 0;
    const int halves = first < m ? 2 * ((m - first + step - 1) / step) : 0, end = g0 + m;
    int qk = 0, pv = 0;                    // next half tile of each product
    bool have_q = false;
    while (pv < halves || seen[0] < end || seen[1] < end) {
      bool moved = false;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int g = seen[v], buf = g & 1;
        if (g < end && test_all(&sm.full[v][buf], (uint32_t)(g / PF_BUFS))) {
          if (step == 2 && ((g - g0 - first) & 1) && (threadIdx.x & 31) == 0) bar_arrive(&sm.empty[v][buf]);
          ++seen[v];
          moved = true;
        }
      }
      if (pv < qk) {  // O += P V of half pv
        const int t = first + step * (pv >> 1), h = pv & 1, g = g0 + t, buf = g & 1;
        if (g < seen[1] && test_all(&p_full[h], done + (uint32_t)(pv >> 1))) {
          tc_after();
          mma_pv(o_col, s_col + 64u * h, v_lo + TILE * (uint32_t)buf + 512u * h, pv > 0);
          tc_commit_to(&pv_done[h]);
          if (h) tc_commit_to(&sm.empty[1][buf]);
          ++pv;
          moved = true;
        }
      }
      if (qk < halves && qk < pv + 2) {  // S = Q K^T of half qk, two ahead of O at most
        const int t = first + step * (qk >> 1), h = qk & 1, g = g0 + t, buf = g & 1;
        if (!have_q) have_q = test_all(&sm.q_full[group], built);
        if (have_q && g < seen[0] && (qk < 2 || test_all(&pv_done[h], done + (uint32_t)(qk >> 1) - 1u))) {
          tc_after();
          mma_qk(s_col + 64u * h, q_lo, k_lo + TILE * (uint32_t)buf + 512u * h);
          tc_commit_to(&s_full[h]);
          if (h) tc_commit_to(&sm.empty[0][buf]);
          ++qk;
          moved = true;
        }
      }
      if (moved) idle = 0;
      else if (++idle > PF_POLL_LIMIT || ((idle & 255u) == 0u && __any_sync(0xffffffffu, *(volatile int*)&sm.fail))) return false;
    }
    done += (uint32_t)(halves >> 1);
    built += halves ? 1u : 0u;
    g0 = end;
    ++pieces;
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
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.bad = 0;
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
// Scores of columns `limit` and up count as -inf.
__device__ __forceinline__ void mask_scores(uint32_t (&s)[32], int limit) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i >= limit) s[i] = 0xFF800000u;
}
// The weights of 32 scores, 2^(ka s + off), as fp16 pairs; their fp32 sums are added to `sum`.
__device__ __forceinline__ void weights(const uint32_t (&s)[32], uint32_t (&w)[16], uint64_t ka2, uint64_t off2, uint64_t (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float e0, e1;
    unpack_f2(fma_f2(pack_f2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), ka2, off2), e0, e1);
    e0 = ex2(e0);
    e1 = ex2(e1);
    sum[i & 1] = add_f2(sum[i & 1], pack_f2(e0, e1));
    w[i] = pack_h2(e0, e1);
  }
}
// The running max has moved: this warp's rows of O are scaled.
__device__ __forceinline__ void scale_o(uint32_t o_col, float f) {
#pragma unroll 1
  for (int x = 0; x < 8; ++x) {
    uint32_t o[16];
    tm_ld16(o_col + 16u * x, o);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
    tm_st16(o_col + 16u * x, o);
  }
}

__device__ __forceinline__ bool softmax_role(const PfArgs& a, PfSmem& sm, Cursor cur, int warp, int lane, uint32_t& copies) {
  const int group = warp >> 2, wq = warp & 3;
  const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
  const uint32_t s_col = sm.tmem + 128u * group + lane_base, o_col = sm.tmem + 256u + 128u * group + lane_base;
  Piece p;
  uint32_t tiles = 0;       // of this group, over all pieces
  copies = 0;               // query operands copied
  int pieces = 0;
  int tg0 = 0;              // tiles of the CTA before this piece
  while (next_piece(a, cur, p)) {
    // (alternating groups also take turns at the first tile, so that two one-tile items overlap)
    const int first = p.dual ? (group + pieces) & 1 : 0;
    const bool some = first < p.m;  // else nothing here waits for the MMAs, and no barrier may move
    if (some && wq == 0 && lane == 0) {
      if (copies == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
      // (the group's MMAs that read the previous operand have finished: pv_done was waited for)
      const RowSet& r = p.own ? a.ro : a.rp;
      const unsigned char* src = q_tile(a, p.own, p.item, p.dual ? 0 : group);
      const int rows = p.dual ? p.rows : min(128, p.rows - 128 * group);
      const uint32_t bytes = (uint32_t)((rows + 7) / 8 * 8) * 128u, dst = smem_addr(sm.q[group]), bar = smem_addr(&sm.q_full[group]);
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
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (!bar_wait(&sm.s_full[group][h], tiles, &sm.fail)) return false;
        // (K tile g cannot be there before V tile g - 4 was, so this barrier is never two phases away)
        if (h == 0 && !bar_wait(&sm.v_info[(tg0 + t) & 3], (uint32_t)((tg0 + t) >> 2), &sm.fail)) return false;
        if (warp_live) {
          tc_after();
          const uint32_t col = s_col + 64u * h;
          uint32_t sa[32], sb[32];
          tm_ld32_async(col, sa);
          tm_ld32_async(col + 32u, sb);
          const PfInfo info = sm.info[(tg0 + t) & 3];
          const PfInfoV iv = sm.info_v[(tg0 + t) & 3];
          const int limit = min(info.nvalid, info.base + info.step * c_of_row) - 64 * h;
          tm_ready64(sa, sb);
          if (__any_sync(0xffffffffu, limit < 64)) {
            mask_scores(sa, limit);
            mask_scores(sb, limit - 32);
          }
          float mx[4] = {minus_inf(), minus_inf(), minus_inf(), minus_inf()};
#pragma unroll
          for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], fmaxf(__uint_as_float(sa[i]), __uint_as_float(sb[i])));
          const float top = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), info.ka, iv.lv);
          // (rows that do not exist hold whatever the operand's memory held: they have no say.  A row's own scores
          // alone move its reference, so its result does not depend on the other rows of the warp)
          const bool up = row < p.rows && top > m + (PF_HEAD + PF_SLACK);
          if (__any_sync(0xffffffffu, up)) {
            const float mn = up ? top - PF_HEAD : m, f = ex2(m - mn);
            m = mn;
            l *= f;
            if (t != first || h) {  // O: once the product before this half's has been added
              if (!bar_wait(&sm.pv_done[group][h ^ 1], h ? tiles : tiles - 1u, &sm.fail)) return false;
              tc_after();
              scale_o(o_col, f);
            }
          }
          const float off = iv.lv - m;
          const uint64_t ka2 = pack_f2(info.ka, info.ka), off2 = pack_f2(off, off);
          uint64_t sum[2] = {0ull, 0ull};
          uint32_t w[16];
          weights(sa, w, ka2, off2, sum);
          tm_st16(col, w);
          weights(sb, w, ka2, off2, sum);
          tm_st16(col + 16u, w);
          float a0, a1;
          unpack_f2(add_f2(sum[0], sum[1]), a0, a1);
          l = fmaf(a0 + a1, iv.iva, l);
          if (limit > iv.vbad - 64 * h) l = __int_as_float(0x7fc00000);  // a value it sees is not finite
          tm_wait_st();
          tc_before();
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&sm.p_full[group][h]);
      }
    }
    // ---- this group's partial of the item ----
    const int hr = p.own ? a.ro.hr : a.rp.hr;
    const int64_t row0 = slot_row(a, p.own, p.item, blockIdx.x);
    const int srow = (p.dual ? group * hr : 128 * group) + 32 * wq + lane;
    if (some && !bar_wait(&sm.pv_done[group][1], tiles - 1u, &sm.fail)) return false;
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
    ++pieces;
  }
  if (copies == 0) asm volatile("griddepcontrol.wait;" ::: "memory");  // (a group without tiles)
  return true;
}

// This CTA gave up, so items may lack table entries and partials (by one thread, behind the query kernel, which
// clears the word).
__device__ __forceinline__ void report_failure(const PfArgs& a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  *(volatile int32_t*)a.bad = 1;
  if (a.status) atomicOr(a.status, 2);
}

template <int MK, int MV, bool DQ>
__global__ void __launch_bounds__(PF_THREADS, 1) prefix_kernel(const __grid_constant__ PfArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  PfSmem& sm = *reinterpret_cast<PfSmem*>(smem_raw);
  // (the swizzle needs 1024-byte aligned tiles; there is no room to align by hand, and no static
  // shared memory that could move the base)
  if (smem_addr(smem_raw) & 1023u) {
    if (threadIdx.x == 0) report_failure(a);
    return;
  }
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  // ---- this CTA's range of the tiles ----
  const int nseg = a.H + (a.ro.rows > 0 ? a.B * a.H : 0);  // (own parts only where they are tiles)
  const int per = (nseg + PF_THREADS - 1) / PF_THREADS;
  long long sum = 0;
  bool short_window = false;
  for (int s = tid * per; s < min(nseg, (tid + 1) * per); ++s) {
    const Seg g = seg_info(a, s);
    const RowSet& r = s >= a.H ? a.ro : a.rp;
    sum += (long long)seg_units(g, r) * r.rt;
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
    for (int r = 0; r < PF_REP; ++r) dst[(r + code) & (PF_REP - 1)] = row;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&sm.q_full[i], 1);
      for (int h = 0; h < 2; ++h) {
        bar_init(&sm.s_full[i][h], 1);
        bar_init(&sm.p_full[i][h], 4);
        bar_init(&sm.pv_done[i][h], 1);
      }
    }
    for (int v = 0; v < 2; ++v)
      for (int i = 0; i < PF_BUFS; ++i) {
        bar_init(&sm.full[v][i], PF_TEAM);
        bar_init(&sm.empty[v][i], 2);
      }
    bar_init(&sm.meet[0], PF_TEAM);
    bar_init(&sm.meet[1], PF_TEAM);
    for (int i = 0; i < 4; ++i) bar_init(&sm.v_info[i], 1);
    bar_init(&sm.drain[0], 1);
    bar_init(&sm.drain[1], 1);
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
  // The counters and caches were there before the whole call; of the kernels before this one only the
  // query tiles are needed, and whoever copies one waits (griddepcontrol.wait) first.  The join may be
  // scheduled from here on and waits for this kernel's end.
  asm volatile("griddepcontrol.launch_dependents;");
  // at least one unit each, so the CTAs with tiles of an item are consecutive
  const long long ctas = min((long long)gridDim.x, total), bid = blockIdx.x;
  if (bid >= ctas) {  // the whole CTA: nothing to do (the kernels before this one still end first)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const long long begin = total * bid / ctas, end = total * (bid + 1) / ctas;
  long long at = before + inc - sum;  // tiles before this thread's segments
  if (at <= begin && begin < at + sum) {
    for (int s = tid * per;; ++s) {
      const RowSet& r = s >= a.H ? a.ro : a.rp;
      const int units = seg_units(seg_info(a, s), r);
      const long long here = (long long)units * r.rt;
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
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sm.tmem)));
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PF_REGS_DECODE));
    ok = warp < 8 + PF_TEAM ? (int)blockIdx.x != a.give_up && decode_role<MK, DQ, false>(a, sm, cur, warp - 8, lane)
                            : decode_role<MV, DQ, true>(a, sm, cur, warp - 8 - PF_TEAM, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PF_REGS_MMA));
    if (warp <= 17) {
      ok = mma_role(a, sm, cur, warp - 16);
      if (!ok) *(volatile int*)&sm.fail = 1;
      // products in flight finish, and their arrivals land, before tensor memory is given back and the CTA ends
      // (whichever role gave up)
      int never = 0;
      tc_commit_to(&sm.drain[warp - 16]);
      if (!bar_wait(&sm.drain[warp - 16], 0u, &never)) ok = false;
    }
  }
  if (!ok) *(volatile int*)&sm.fail = 1;
  __syncwarp();
  tc_before();
  __syncthreads();
  if (tid == 0 && *(volatile int*)&sm.fail) report_failure(a);
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
__device__ __forceinline__ void join_item(const PfArgs& a, bool own, int seg, int tiles, int row, int wi, int lane, float& m, float& l, float (&v)[4]) {
  const RowSet& r = own ? a.ro : a.rp;
  const int64_t item = (int64_t)(own ? seg - a.H : seg) * r.rt + row / 256;
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
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wi = warp % WPR;
  const int64_t r = ((int64_t)blockIdx.x * JOIN_WARPS + warp) / WPR;  // (b, c, head)
  const int nh = a.H * a.G;
  const bool live = r < (int64_t)a.B * a.C * nh;
  float2 own = make_float2(NEG_BIG, 0.f);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = NEG_BIG, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
  const int hq = (int)(r % nh), bc = (int)(r / nh), c = bc % a.C, b = bc / a.C, h = hq / a.G, gi = hq % a.G;
  int tiles_p = 0, tiles_o = 0;
  if (live) {  // (the counters were there before the whole call)
    tiles_p = seg_info(a, h).tiles;
    tiles_o = a.own_lse ? 0 : seg_info(a, a.H + b * a.H + h).tiles;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (*a.bad) {
    l = __int_as_float(0x7fc00000);
  } else if (live) {
    if (a.own_lse && wi == 0) {
      own = a.own_lse[r];
      o = *reinterpret_cast<const float4*>(a.own_out + r * D + 4 * lane);
    }
    join_item<WPR>(a, false, h, tiles_p, (b * a.C + c) * a.G + gi, wi, lane, m, l, v);
    if (!a.own_lse) join_item<WPR>(a, true, a.H + b * a.H + h, tiles_o, c * a.G + gi, wi, lane, m, l, v);
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
  // a value that is not finite makes the whole row NaN: own rows of the decode kernel, whose window values keep their
  // dims, as those of the tiles
  const float odd = fmaf(v[0], 0.f, fmaf(v[1], 0.f, fmaf(v[2], 0.f, v[3] * 0.f)));  // 0, or NaN
  if (__any_sync(0xffffffffu, odd != 0.f)) v[0] = v[1] = v[2] = v[3] = __int_as_float(0x7fc00000);
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
  // (measured: 5 against 3, 8 x 128 queries behind 32k, 662 against 791 us; where the groups alternate
  // tiles two items overlap, and 3 against 5 and 1: 64 queries behind 131k, 251 against 258 and 298 us)
  r.cost = rows > 128 ? 5 : 3;
  return r;
}

// With one query per sequence the own part has 1 to 8 rows per (b, kv-head), which a 128-row tile
// wastes; the decode kernel reads such a cache faster, but has a fixed cost (its window is one warp's
// work).  Measured, 8 kv-heads, 4 queries each, whole call behind an 8k prefix, tiles against decode
// kernel: 16 x 300 own tokens 42 / 66 us, 16 x 1200 56 / 55, 16 x 2200 65 / 55; 64 x 128 74 / 113,
// 64 x 200 83 / 84, 64 x 300 93 / 76, 64 x 2200 213 / 106.  The lengths are on the device: the capacity
// decides.
bool own_by_decode(int n_queries, int B, int H, int own_capacity) {
  return n_queries == 1 && (int64_t)B * H * (own_capacity / BLK + 4) > 2800;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: (own part by decode: its workspace, whose counters come first, then its rows and their
// denominators), the query tiles, the item table, the (m, l) pairs and the sums of every slot.
struct PfLayout {
  RowSet rp, ro;
  size_t own_out, own_lse, qt, tab, ml, acc, bytes;
};
PfLayout layout(int B, int H, int g, int C, int own_capacity) {
  PfLayout y;
  const bool dec = own_by_decode(C, B, H, own_capacity);
  y.rp = row_set((int64_t)B * C * g);
  y.ro = row_set(dec ? 0 : (int64_t)C * g);
  const int64_t ip = (int64_t)H * y.rp.rt, io = (int64_t)B * H * y.ro.rt, rows_out = (int64_t)B * C * H * g;
  const int64_t rows = (ip + PF_CTAS) * 2 * y.rp.hr + (io + PF_CTAS) * 2 * y.ro.hr;
  // (the counters' place is kept for any C, so that one zero-filled workspace serves calls of several)
  y.own_out = up256(dec ? decode_workspace_bytes(B, H, decode_geometry(B, own_capacity, H * g, H)) : decode_counter_bytes(B, H));
  y.own_lse = y.own_out + (dec ? up256((size_t)rows_out * D * sizeof(float)) : 0);
  y.qt = y.own_lse + (dec ? up256((size_t)rows_out * sizeof(float2)) : 0);
  y.tab = y.qt + up256((size_t)(ip * 2 * q_tile_bytes(y.rp) + io * 2 * q_tile_bytes(y.ro)));
  y.ml = y.tab + up256((size_t)(ip + io + 1) * sizeof(int2));  // (and the failure word)
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
  const size_t smem = sizeof(PfSmem);
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
                          int give_up, cudaStream_t s) {
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
  a.bad = reinterpret_cast<int32_t*>(a.tab + (int64_t)a.H * y.rp.rt + (int64_t)a.B * a.H * y.ro.rt);
  a.give_up = give_up;
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
  if (own_by_decode(a.C, a.B, a.H, k.capacity)) {
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

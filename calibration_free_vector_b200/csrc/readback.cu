// Reading a compressed cache back (sm_100a): every token of [start, start + n) as an
// ordinary row of fp32, bf16 or fp16.
//
// For a quantized token t of block b, with H the orthonormal Hadamard matrix,
//   x_hat = H ((u_hat s2 + o_b) s1) = ((H u_hat) s2 + H o_b) s1        (H^T = H),
// so H is applied to the codewords themselves, which are exact in fp16, and the norms
// enter in fp32 afterwards; H o_b is formed once per unit of work.
//
// The transform is the one of hadamard_mma.cuh (M = the 16 tokens of a tile).  Its A operand,
// for each r the 16 values of sub-vectors 2r and 2r + 1, is gathered by ldmatrix straight from an
// 8-fold replicated fp16 codebook, the stored signs XOR-ed on.  A lane ends with four consecutive
// dims of a row: 8- or 16-byte stores, every 32-byte sector written whole.
//
// Bytes bound it: a 2-bit token is 38 bytes read and 256 (bf16) written.  Measured on 16 x 8 x 32768
// 2-bit tokens to bf16: 279-284 us, 4.3-4.4 TB/s, 66-67 % of the copy bandwidth; DRAM traffic is the
// 1.18 GB that it has to be.  Warps wait for their reads behind the stores' traffic.  Measured and not
// kept: rows sent through shared memory by one bulk copy each (275 us) or by stores of two whole rows
// (259, ragged batches slower), reads two tiles ahead (257, ragged batches slower).

#include "hadamard_mma.cuh"
#include "nsn_launch.h"

namespace nsn {
namespace {

constexpr int RB_WARPS = 8;
constexpr int RB_CTAS = 2;  // resident per SM (registers)
constexpr float RB_INV_SQRT_D = 0.08838834764831845f;  // 1/sqrt(128)

struct RbSmem {
  alignas(128) uint4 cb[NCODES][8];  // codeword c, replica r at byte 128 c + 16 r: eight ldmatrix rows, eight bank groups
  alignas(16) float ho[RB_WARPS][D];  // H o of the unit's block
};

__device__ __forceinline__ uint32_t rb_pack(float x, float y, int dt) {
  if (dt == NSN_DTYPE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four consecutive elements of an output row; nothing here is read again, so the
// stores are marked to leave the L2 first.
template <int DT>
__device__ __forceinline__ void rb_store4(void* out, int64_t off, float a, float b, float c, float d) {
  if constexpr (DT == NSN_DTYPE_F32) {
    __stcs(reinterpret_cast<float4*>(static_cast<float*>(out) + off), make_float4(a, b, c, d));
  } else {
    __stcs(reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + off), make_uint2(rb_pack(a, b, DT), rb_pack(c, d, DT)));
  }
}

// What a lane reads of one 16-token tile: the 8 codes of its ldmatrix row (token
// (l & 7) + 8 ((l >> 3) & 1), sub-vectors of parity l >> 4), the sign words and norms of
// tokens g and g + 8.
struct RbTile {
  uint2 code;
  uint32_t sign[2];
  uint32_t norm[2], level[2];  // fp16 (s1, s2); or fp16 s2, and the byte with the s1 level
};

template <int MODE, bool DQ>
__device__ __forceinline__ void rb_load(RbTile& tl, const CacheView& cv, int64_t seq, int t0, int lane) {
  const int g = lane >> 2, p = lane & 3;
  const int64_t base = seq * (int64_t)cv.capacity + t0;
  const int tok = (lane & 7) + 8 * ((lane >> 3) & 1);
  tl.code = ld_v2(cv.codes + (base + tok) * NSUB + 8 * (lane >> 4));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t t = base + g + 8 * i;
    if constexpr (MODE == NSN_MODE_2BIT)
      tl.sign[i] = ld_u32(cv.signs + t * NSUB + 4 * p);
    if constexpr (DQ) {
      tl.level[i] = ld_u8(cv.s1_levels + (t >> 1));
      tl.norm[i] = ld_u16(reinterpret_cast<const __half*>(cv.norms) + t);
    } else {
      tl.norm[i] = ld_u32(cv.norms + t);
    }
  }
}

// One warp = one unit: `unit_tiles` consecutive 16-token tiles of one block of one
// sequence.  A tile that crosses the quantized part's end, or the range's ends, loads
// whole (the buffers hold whole blocks) and stores the rows that exist.
template <int MODE, bool DQ, int DT>
__global__ void __launch_bounds__(32 * RB_WARPS, RB_CTAS)
readback_kernel(CacheView cv, int start, int n_tokens, const float* __restrict__ cb, void* __restrict__ out, int64_t sb,
                int64_t st, int64_t sh, int unit_tiles, int units_per_seq, int64_t n_units) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  RbSmem& sm = *reinterpret_cast<RbSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, p = lane & 3;
  static_assert(32 * RB_WARPS == NCODES, "one codeword per thread");
  {
    float c[SUB];
    load8<NSN_DTYPE_F32>(cb, (int64_t)tid * SUB, c);
    const uint4 row = pack8_f16(c);
#pragma unroll
    for (int r = 0; r < 8; ++r) sm.cb[tid][(r + tid) & 7] = row;
  }
  __syncthreads();
  const uint32_t cb_base = smem_addr(&sm.cb[0][0]) + (uint32_t)(lane & 7) * 16u;

  uint32_t hb[2][2];
  h16_operand(hb, lane);

  const int unit_tok = 16 * unit_tiles;
  const int first_unit = start / unit_tok;
  for (int64_t unit = (int64_t)blockIdx.x * RB_WARPS + warp; unit < n_units; unit += (int64_t)gridDim.x * RB_WARPS) {
    // the heads of one token range are consecutive units: with rows [B, T, H, 128] they write one
    // contiguous stretch of memory at about the same time
    const int64_t bu = unit / cv.n_kv_heads;
    const int64_t seq = bu / units_per_seq * cv.n_kv_heads + unit % cv.n_kv_heads;
    const int u0 = (first_unit + (int)(bu % units_per_seq)) * unit_tok;  // first token of the unit
    const int nq = max(0, min(cv.n_quant[seq], cv.capacity));
    const int nw = cv.window_len > 0 ? max(0, min(cv.n_window[seq], cv.window_len)) : 0;
    const int lo = max(u0, start), hi = min(u0 + unit_tok, min(start + n_tokens, nq + nw));
    if (lo >= hi) continue;
    const int b = (int)(seq / cv.n_kv_heads), h = (int)(seq % cv.n_kv_heads);
    const int64_t row0 = (int64_t)b * sb + (int64_t)h * sh - (int64_t)start * st;  // row of token t at row0 + t st
    const int qhi = min(hi, nq);
    if (lo < qhi) {
      const int64_t blk = seq * (int64_t)(cv.capacity / BLK) + u0 / BLK;
      float2 s1_ls = make_float2(0.f, 0.f), o_ls = make_float2(0.f, 0.f);
      if constexpr (DQ) {
        const uint2 par = *reinterpret_cast<const uint2*>(cv.dq_params + blk * 8);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&par.x));
        const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&par.y));
        s1_ls = make_float2(a.x, (a.y - a.x) / 15.0f);
        o_ls = make_float2(c.x, (c.y - c.x) / 15.0f);
      }
      const int tb = u0 + ((lo - u0) & ~15);
      RbTile next;
      rb_load<MODE, DQ>(next, cv, seq, tb, lane);
      // H o of the block: the mean row as every token of one tile (fp16 hi + lo parts when it
      // is read back from levels; an fp16 mean row is its own hi part)
      {
        float E[8][2][4];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          uint32_t hi2[2], lo2[2] = {0u, 0u};
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const int d = 16 * r + 8 * kk + 2 * p;
            if constexpr (DQ) {
              const uint32_t two = reinterpret_cast<const uint8_t*>(cv.means)[blk * (D / 2) + d / 2];
              split_half2(fmaf((float)(two & 15u), o_ls.y, o_ls.x), fmaf((float)(two >> 4), o_ls.y, o_ls.x), hi2[kk], lo2[kk]);
            } else {
              hi2[kk] = *reinterpret_cast<const uint32_t*>(cv.means + blk * D + d);
            }
          }
          const uint32_t ah[4] = {hi2[0], hi2[0], hi2[1], hi2[1]}, al[4] = {lo2[0], lo2[0], lo2[1], lo2[1]};
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            E[r][nt][0] = E[r][nt][1] = E[r][nt][2] = E[r][nt][3] = 0.f;
            h16_mma(E[r][nt], ah, hb[nt]);
            if constexpr (DQ) h16_mma(E[r][nt], al, hb[nt]);
          }
        }
        h8_butterflies(E);
        __syncwarp();  // the previous unit's rows are written
        if (g == 0) {
#pragma unroll
          for (int r = 0; r < 8; ++r)
            *reinterpret_cast<float4*>(&sm.ho[warp][16 * r + 4 * p]) = make_float4(E[r][0][0], E[r][0][1], E[r][1][0], E[r][1][1]);
        }
        __syncwarp();
      }
      for (int t0 = tb; t0 < qhi; t0 += 16) {
        const RbTile cur = next;
        if (t0 + 16 < qhi) rb_load<MODE, DQ>(next, cv, seq, t0 + 16, lane);
        float E[8][2][4];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const uint32_t code = __byte_perm(r < 4 ? cur.code.x : cur.code.y, 0u, 0x4440u | (uint32_t)(r & 3));
          uint32_t a[4];
          ldsm_x4(cb_base + code * 128u, a);
          if constexpr (MODE == NSN_MODE_2BIT) {
            a[0] ^= (cur.sign[0] << (2 * r)) & 0x80008000u;
            a[1] ^= (cur.sign[1] << (2 * r)) & 0x80008000u;
            a[2] ^= (cur.sign[0] << (2 * r + 1)) & 0x80008000u;
            a[3] ^= (cur.sign[1] << (2 * r + 1)) & 0x80008000u;
          }
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            E[r][nt][0] = E[r][nt][1] = E[r][nt][2] = E[r][nt][3] = 0.f;
            h16_mma(E[r][nt], a, hb[nt]);
          }
        }
        h8_butterflies(E);
        const int t = t0 + g;
        const bool have[2] = {t >= lo && t < qhi, t + 8 >= lo && t + 8 < qhi};
        const int64_t off = row0 + (int64_t)t * st + 4 * p;
        uint64_t s1[2], s2[2];  // s1 / sqrt(128) and s2 of the two tokens, for two columns at once
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2 n = __half22float2(*reinterpret_cast<const __half2*>(&cur.norm[i]));
          if constexpr (DQ) n = make_float2(fmaf((float)((cur.level[i] >> (4 * (g & 1))) & 15u), s1_ls.y, s1_ls.x), n.x);
          s1[i] = pack_f2(n.x * RB_INV_SQRT_D, n.x * RB_INV_SQRT_D);
          s2[i] = pack_f2(n.y, n.y);
        }
        const uint64_t zero = pack_f2(0.f, 0.f);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float4 ho = *reinterpret_cast<const float4*>(&sm.ho[warp][16 * r + 4 * p]);
          const uint64_t h01 = pack_f2(ho.x, ho.y), h23 = pack_f2(ho.z, ho.w);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v[4];  // ((H u_hat) s2 + H o) s1
            unpack_f2(fma_f2(fma_f2(pack_f2(E[r][0][2 * i], E[r][0][2 * i + 1]), s2[i], h01), s1[i], zero), v[0], v[1]);
            unpack_f2(fma_f2(fma_f2(pack_f2(E[r][1][2 * i], E[r][1][2 * i + 1]), s2[i], h23), s1[i], zero), v[2], v[3]);
            if (have[i]) rb_store4<DT>(out, off + 8 * i * st + 16 * r, v[0], v[1], v[2], v[3]);
          }
        }
      }
    }
    // window rows, as they are: four reads in flight
#pragma unroll 1
    for (int t0 = max(lo, nq); t0 < hi; t0 += 4) {
      uint2 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < hi)
          x[i] = ld_v2(cv.window + (seq * cv.window_len + (t0 + i - nq)) * (int64_t)D + 4 * lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < hi) {
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x[i].x));
          const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&x[i].y));
          rb_store4<DT>(out, row0 + (int64_t)(t0 + i) * st + 4 * lane, a.x, a.y, c.x, c.y);
        }
    }
  }
}

template <int MODE, bool DQ, int DT>
cudaError_t launch_t(const CacheView& cv, int start, int n_tokens, const float* cb, void* out, int64_t sb, int64_t st,
                     int64_t sh, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t nseq = (int64_t)cv.batch * cv.n_kv_heads, ctas = (int64_t)sms * RB_CTAS;
  // A whole block per unit forms H o once per 128 tokens; units are made smaller until every resident
  // warp has four, so that ragged lengths even out (128 ragged sequences of up to 4002 tokens: 31 us,
  // with one unit per warp 39; 8 sequences of 4096, host-bound either way).
  int unit_tiles = BLK / 16;
  const int64_t end = (int64_t)start + n_tokens;
  const auto per_seq = [&](int tiles) { return (end + 16 * tiles - 1) / (16 * tiles) - start / (16 * tiles); };
  while (unit_tiles > 1 && nseq * per_seq(unit_tiles) < 4 * ctas * RB_WARPS) unit_tiles >>= 1;
  const int64_t ups = per_seq(unit_tiles), n_units = nseq * ups;
  const int64_t want = (n_units + RB_WARPS - 1) / RB_WARPS;
  readback_kernel<MODE, DQ, DT><<<(unsigned)(want < ctas ? want : ctas), 32 * RB_WARPS, sizeof(RbSmem), s>>>(
      cv, start, n_tokens, cb, out, sb, st, sh, unit_tiles, (int)ups, n_units);
  return cudaGetLastError();
}

template <int MODE, bool DQ>
cudaError_t launch_m(const CacheView& cv, int start, int n, const float* cb, void* out, int dtype, int64_t sb, int64_t st,
                     int64_t sh, cudaStream_t s) {
  switch (dtype) {
    case NSN_DTYPE_F32: return launch_t<MODE, DQ, NSN_DTYPE_F32>(cv, start, n, cb, out, sb, st, sh, s);
    case NSN_DTYPE_BF16: return launch_t<MODE, DQ, NSN_DTYPE_BF16>(cv, start, n, cb, out, sb, st, sh, s);
    default: return launch_t<MODE, DQ, NSN_DTYPE_F16>(cv, start, n, cb, out, sb, st, sh, s);
  }
}

}  // namespace

cudaError_t launch_readback(const CacheView& cv, int start, int n_tokens, const float* cb, void* out, int dtype, int64_t sb,
                            int64_t st, int64_t sh, cudaStream_t s) {
  if (cv.mode == NSN_MODE_2BIT)
    return cv.dq ? launch_m<NSN_MODE_2BIT, true>(cv, start, n_tokens, cb, out, dtype, sb, st, sh, s)
                 : launch_m<NSN_MODE_2BIT, false>(cv, start, n_tokens, cb, out, dtype, sb, st, sh, s);
  return cv.dq ? launch_m<NSN_MODE_1BIT, true>(cv, start, n_tokens, cb, out, dtype, sb, st, sh, s)
               : launch_m<NSN_MODE_1BIT, false>(cv, start, n_tokens, cb, out, dtype, sb, st, sh, s);
}

}  // namespace nsn

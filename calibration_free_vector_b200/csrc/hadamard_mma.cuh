// The 128-point Hadamard transform of 16 rows on the tensor cores (warp level, sm_100a).
//
// H of 128 values is the Kronecker product H8 (x) H16 (Sylvester order).  With dim d = 16 r + c,
// the H16 factor is, for each r, the 16 rows' values of that r (M = 16, K = 16) times a 16 x 16
// matrix of +-1, and the H8 factor three butterfly stages over r, which are register additions
// because a lane holds all eight r of its (row, column)s.  Against the warp-shuffle transform
// this has no exchange between lanes at all.  Sums are fp32; +-1 is exact, so fp16 inputs (or
// fp16 hi + lo parts) lose nothing.
//
// The columns of H16 are dealt to the two n-tiles so that lane (g, p) = (lane / 4, lane % 4)
// ends with four consecutive dims 16 r + 4 p .. + 3 of rows g and g + 8:
//   row g:     E[r][0][0], E[r][0][1], E[r][1][0], E[r][1][1]
//   row g + 8: E[r][0][2], E[r][0][3], E[r][1][2], E[r][1][3].
#pragma once

#include "nsn_common.cuh"

namespace nsn {

// B fragments of H16: rows k = 2p, 2p + 1 (+ 8), column c of each n-tile's column g.
__device__ __forceinline__ void h16_operand(uint32_t (&hb)[2][2], int lane) {
  const int g = lane >> 2, p = lane & 3;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const int c = 4 * (g >> 1) + 2 * nt + (g & 1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int k = 2 * p + 8 * kk;
      const uint32_t lo = (__popc(k & c) & 1) ? 0xBC00u : 0x3C00u, hi = (__popc((k + 1) & c) & 1) ? 0xBC00u : 0x3C00u;
      hb[nt][kk] = lo | (hi << 16);
    }
  }
}

// d += A (16 rows x 16) * B (16 x 8), fp16 operands, fp32 sums.
__device__ __forceinline__ void h16_mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The H8 factor: butterflies over r, two columns per instruction.
__device__ __forceinline__ void h8_butterflies(float (&E)[8][2][4]) {
  uint64_t e[8][2][2];
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) e[r][nt][i] = pack_f2(E[r][nt][2 * i], E[r][nt][2 * i + 1]);
  const uint64_t minus = pack_f2(-1.f, -1.f);
#pragma unroll
  for (int step = 1; step < 8; step <<= 1)
#pragma unroll
    for (int a = 0; a < 8; ++a)
      if (!(a & step))
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint64_t u = e[a][nt][i], w = e[a + step][nt][i];
            e[a][nt][i] = add_f2(u, w);
            e[a + step][nt][i] = fma_f2(w, minus, u);  // u - w (the product is exact)
          }
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) unpack_f2(e[r][nt][i], E[r][nt][2 * i], E[r][nt][2 * i + 1]);
}

}  // namespace nsn

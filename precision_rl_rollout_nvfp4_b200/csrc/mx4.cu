// MXFP4: quantization, the values of a quantized tensor, and both at once.
//
// A block is 32 consecutive elements along K.  With the block's largest
// magnitude a (from the bits of its elements), E = floor(log2 a) - 2 clamped
// to [-127, 127] (-127 for an all-zero block), so a / 2^E is in [4, 8) and the
// largest E2M1 value, 6 = 1.5 2^2, has the same exponent; code = E2M1(x 2^-E),
// nearest, ties to the even code, saturating at 6, the sign of x kept.  A
// block with an infinity or a NaN gets scale 255 (NaN) and codes 0, so that
// each of its values reads back as NaN and every product that touches it is
// NaN.  x 2^-E is exact: the factor is a power of two and a result below
// 2^-126 is code 0 in any rounding.
#include "mx4.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

// Scale word (4 blocks) of (row, 128-element atom) in the tiled layout.
__device__ __forceinline__ int64_t tiled_word(int64_t row, int64_t atom, int64_t atoms) {
  return ((row >> 7) * atoms + atom) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4;
}

// 32 bytes to or from memory: one 256-bit access where the address allows it
// (WIDE), two of 16 bytes otherwise.
template <bool WIDE>
__device__ __forceinline__ void load32(const void* p, uint32_t (&v)[8]) {
  if constexpr (WIDE) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
  } else {
    const uint4 a = *static_cast<const uint4*>(p), b = static_cast<const uint4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// The units a warp takes, 512 elements (four atoms) of one row each, in row
// order; the position is the same in all its lanes (uniform registers) and
// moves on without a division.
struct Units {
  int64_t u, end, step, row;
  uint32_t seg, drow, dseg, segs;
  __device__ Units(int64_t rows, uint32_t n) : segs(n) {
    const int64_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
    u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp;
    step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    end = rows * n;
    row = u / n;
    seg = static_cast<uint32_t>(u - row * n);
    drow = static_cast<uint32_t>(step / n);
    dseg = static_cast<uint32_t>(step - static_cast<int64_t>(drow) * n);
  }
  __device__ __forceinline__ bool more() const { return u < end; }
  __device__ __forceinline__ void next() {
    u += step;
    row += drow;
    seg += dseg;
    if (seg >= segs) {
      seg -= segs;
      ++row;
    }
  }
};

// The larger magnitude of each half, NaN if either is (its sign means nothing).
__device__ __forceinline__ uint32_t bf16x2_absmax(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The eight E2M1 codes of a word as bf16 pairs.  A code's three magnitude bits
// index two tables of eight bytes (the halves of the bf16 of 0, 0.5, 1, 1.5,
// 2, 3, 4, 6), four codes per byte permutation; with the sign bit set the
// permutation replicates the sign of the byte it picks, which makes the mask.
__device__ __forceinline__ void e2m1x8_bf16(uint32_t codes, uint32_t* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = codes >> (16 * h), sel = c & 0x7777u;
    uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel);
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    uint32_t neg;                                          // 0xFF for a negative code, 0x80 otherwise
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(neg) : "r"(0x80808080u), "r"(c));
    hi |= ((neg & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    v[2 * h] = __byte_perm(lo, hi, 0x5140);
    v[2 * h + 1] = __byte_perm(lo, hi, 0x7362);
  }
}

// 2^E of a scale byte as a bf16 pair (255: NaN; 0: 2^-127, subnormal).  A
// product with an E2M1 value has two significant bits and at least 2^-128, so
// it is exact.
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t sb) {
  const uint32_t b = sb == 255u ? 0x7FC0u : (sb ? sb << 7 : 0x0040u);
  return b | (b << 16);
}

// A lane takes 16 elements, two lanes a block, eight an atom.  Rows and blocks
// of the padding get scale 0 (tiled layout).
//
// 2 bytes read and 17/32 (or with QDQ 2 more) written per element.  The
// integer pipe is nearly as busy as memory (with a division and 64-bit
// addresses per lane and 8 elements it was the bound: 88 us for 32768 x 4096),
// hence the uniform positions and one address per 32 bytes.
template <bool CODES, bool QDQ, bool WIDE>
__global__ void __launch_bounds__(kThreads)
mx4_quant_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t prows, uint32_t K, int64_t ldx, uint32_t segs,
                 uint32_t atoms, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int layout,
                 uint16_t* __restrict__ qdq, int64_t ldo) {
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t lane = threadIdx.x & 31, sub = lane & 7;
  for (Units it(prows, segs); it.more(); it.next()) {
    const int64_t row = it.row;
    const uint32_t col = it.seg * 512 + 16 * lane;
    const bool in = row < rows && col < K;                    // K % 32 == 0: a block is in or out
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in && NV_IDX(in_matrix(row, col, 16, rows, K, ldx))) load32<WIDE>(x + row * ldx + col, w);
    uint32_t m2 = bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(w[0], w[1]), bf16x2_absmax(w[2], w[3])),
                                bf16x2_absmax(bf16x2_absmax(w[4], w[5]), bf16x2_absmax(w[6], w[7])));
    m2 = bf16x2_absmax(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, 1));         // the block's other half
    m2 &= 0x7FFF7FFFu;
    const uint32_t field = max(m2 & 0xFFFFu, m2 >> 16) >> 7;  // exponent field of the largest magnitude
    const bool bad = field == 255u;
    const uint32_t sb = bad ? 255u : (field > 2u ? field - 2u : 0u);     // E + 127
    const float inv = __uint_as_float((254u - (bad ? 0u : sb)) << 23);   // 2^-E
    const uint64_t inv2 = f2_pack(inv, inv);
    uint32_t out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint64_t p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = f2_mul(bf16x2_to_f2(w[4 * h + j]), inv2);
      out[h] = bad ? 0u : e2m1x8_f2(p);
    }
    if (CODES) {
      if (in && NV_IDX(in_matrix(row, col / 2, 8, rows, K / 2, K / 2)))
        *reinterpret_cast<uint2*>(codes + row * (K / 2) + col / 2) = make_uint2(out[0], out[1]);
      if (layout == 1) {
        // the four blocks' scales of an atom as one word
        uint32_t word = in ? sb << (8 * (sub >> 1)) : 0u;
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
        const uint32_t atom = it.seg * 4 + (lane >> 3);
        if (sub == 0 && atom < atoms && NV_IDX(tiled_word(row, atom, atoms) + 4 <= scale_extent(rows, K, 1, 32)))
          *reinterpret_cast<uint32_t*>(scales + tiled_word(row, atom, atoms)) = word;
      } else if (in && (lane & 1) == 0 && NV_IDX(in_matrix(row, col / 32, 1, rows, K / 32, K / 32))) {
        scales[row * (K / 32) + col / 32] = static_cast<uint8_t>(sb);
      }
    }
    if (QDQ && in && NV_IDX(in_matrix(row, col, 16, rows, K, ldo))) {
      const uint32_t s = scale_bf16x2(sb);
      uint32_t v[8];
      e2m1x8_bf16(out[0], v);
      e2m1x8_bf16(out[1], v + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = bf16x2_mul(v[j], s);
      store32<WIDE>(qdq + row * ldo + col, v);
    }
  }
}

// Values of an MXFP4 tensor: 17/32 bytes read, 2 or 4 written per element;
// bound by the writes (filling the same buffer takes 69 us for 32768 x 4096
// bf16).
template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(kThreads)
mx4_dequant_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int layout, int64_t rows,
                   uint32_t K, uint32_t segs, uint32_t atoms, void* __restrict__ y, int64_t ldy) {
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t lane = threadIdx.x & 31;
  for (Units it(rows, segs); it.more(); it.next()) {
    const int64_t row = it.row;
    const uint32_t col = it.seg * 512 + 16 * lane;
    if (col >= K) continue;
    if (!NV_IDX(in_matrix(row, col / 2, 8, rows, K / 2, K / 2) && in_matrix(row, col, 16, rows, K, ldy))) continue;
    const uint2 c = *reinterpret_cast<const uint2*>(codes + row * (K / 2) + col / 2);
    const int64_t off = layout == 1 ? tiled_word(row, it.seg * 4 + (lane >> 3), atoms) + ((lane & 7) >> 1)
                                    : row * (K / 32) + col / 32;
    const uint32_t s = scale_bf16x2(NV_IDX(off < scale_extent(rows, K, layout, 32)) ? scales[off] : 255u);
    uint32_t v[8];
    e2m1x8_bf16(c.x, v);
    e2m1x8_bf16(c.y, v + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = bf16x2_mul(v[j], s);
    if (BF16) {
      store32<WIDE>(static_cast<uint16_t*>(y) + row * ldy + col, v);
    } else {                                                 // bf16 bits widen to fp32
      float* dst = static_cast<float*>(y) + row * ldy + col;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = v[4 * h + j] << 16;
          f[2 * j + 1] = v[4 * h + j] & 0xFFFF0000u;
        }
        store32<WIDE>(dst + 8 * h, f);
      }
    }
  }
}

unsigned grid_for(int64_t units) {
  const int64_t ctas = (units + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  return static_cast<unsigned>(ctas < cap ? ctas : cap);
}

bool aligned32(const void* p, int64_t ld_bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && ld_bytes % 32 == 0;
}

template <bool CODES, bool QDQ>
cudaError_t quant(bool wide, int64_t units, cudaStream_t s, const uint16_t* x, int64_t rows, int64_t prows, int64_t K,
                  int64_t ldx, uint32_t segs, uint32_t atoms, uint8_t* codes, uint8_t* scales, int layout,
                  uint16_t* qdq, int64_t ldo) {
  return launch_k(wide ? mx4_quant_kernel<CODES, QDQ, true> : mx4_quant_kernel<CODES, QDQ, false>,
                  dim3(grid_for(units)), dim3(kThreads), 0, s, nullptr, 0, x, rows, prows, static_cast<uint32_t>(K), ldx,
                  segs, atoms, codes, scales, layout, qdq, ldo);
}

}  // namespace

cudaError_t launch_mx4_quant(const uint16_t* x, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                             uint8_t* scales, int layout, uint16_t* qdq, int64_t ldo, cudaStream_t s) {
  const uint32_t segs = static_cast<uint32_t>((K + 511) / 512), atoms = static_cast<uint32_t>((K + 127) / 128);
  // the tiled layout's padding rows are units too (they write zero scales)
  const int64_t prows = codes != nullptr && layout == 1 ? (rows + 127) / 128 * 128 : rows;
  const int64_t units = prows * segs;
  if (units == 0) return cudaSuccess;
  const bool wide = aligned32(x, 2 * ldx) && (qdq == nullptr || aligned32(qdq, 2 * ldo));
  const cudaError_t e =
      codes == nullptr
          ? quant<false, true>(wide, units, s, x, rows, prows, K, ldx, segs, atoms, codes, scales, layout, qdq, ldo)
      : qdq == nullptr
          ? quant<true, false>(wide, units, s, x, rows, prows, K, ldx, segs, atoms, codes, scales, layout, qdq, ldo)
          : quant<true, true>(wide, units, s, x, rows, prows, K, ldx, segs, atoms, codes, scales, layout, qdq, ldo);
  return e;
}

cudaError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int layout, int64_t rows, int64_t K,
                               void* y, int y_dtype, int64_t ldy, cudaStream_t s) {
  const uint32_t segs = static_cast<uint32_t>((K + 511) / 512), atoms = static_cast<uint32_t>((K + 127) / 128);
  const int64_t units = rows * segs;
  if (units == 0) return cudaSuccess;
  const bool wide = aligned32(y, ldy * (y_dtype == 1 ? 2 : 4));
  auto k = y_dtype == 1 ? (wide ? mx4_dequant_kernel<true, true> : mx4_dequant_kernel<true, false>)
                        : (wide ? mx4_dequant_kernel<false, true> : mx4_dequant_kernel<false, false>);
  const cudaError_t e = launch_k(k, dim3(grid_for(units)), dim3(kThreads), 0, s, nullptr, 0, codes, scales, layout, rows,
                                 static_cast<uint32_t>(K), segs, atoms, y, ldy);
  return e;
}

NV_DEFINE_BOUNDS_READER(bounds_flags_mx4)

}  // namespace nvfp4

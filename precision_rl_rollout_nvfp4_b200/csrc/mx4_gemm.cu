// MXFP4 products on the 5th-generation tensor cores (tcgen05 kind::mxf4, one
// UE8M0 scale per 32 elements, fp32 accumulators in TMEM):
//
//     Y = X W^T                              (plain)
//     Y = act(X W^T) * (X Up^T)              (gated: both projections, the
//                                             activation and the product)
//
// with Y as fp32, bf16, or quantized to MXFP4 in the epilogue (the operand of
// the down projection: the gated values never reach memory wider than 4 bits).
// The epilogue works on the fp32 accumulators; Y is rounded once.
#include "mx4_common.cuh"

namespace nvfp4 {
namespace {

using namespace umma;

constexpr int kTile = 128;                       // weight rows of a tile (TMEM lanes)
constexpr int kWTile = kTile * kRowBytes;        // 16 KB: 128 rows x 256 codes
constexpr int kThreads = 224;                    // warps: 0 loads, 1 MMA, 2..5 epilogue, 6 spare

// ---------------------------------------------------------------------------
// Few tiles: NT tokens (16, 32 or 64) x 128 weight rows.  The weight rows are
// the MMA's M side and the tokens its N side, so a single token costs one 128 x
// 16 product per 128 weight rows instead of a 128-row activation tile that is
// nearly empty.  The time is that of reading the weights once and a fixed 3 us
// (launch, first load, last product, reduction): one token, cold weights, 4096
// -> 11008 6.5 us where the 24 MB alone take 3.7; gated 10.6 where 48 MB take
// 7.3.  More loads in flight, sequential prefetches of the rows, or the
// next kernel's weights brought into L2 on the way did not shorten it.
//
// A cluster of S CTAs (up to 8) shares a tile, split over K, so that all SMs read.  Each
// CTA owns a share of the tokens, in quads: every CTA writes its fp32 partials
// of a token into the owner's shared memory and arrives on its barrier; the
// owner adds the S partials in CTA order.  (Reading the partials from their
// CTAs instead took S dependent remote loads of 0.2 us and a second barrier:
// 10.6 us for 16 tokens at 4096 x 4096, now 5.0.)
//
// XQ: X is bf16 and each CTA quantizes the rows of its K steps itself (the
// epilogue warps, idle until the end), straight into the operand tile: one
// launch and one pass over X fewer than quantizing first.
//
// Per SM either two CTAs (shared memory of at most 113 KB, 256 TMEM columns
// each; three do not fit) or one (more than 113 KB): no CTA ever waits for
// TMEM that another CTA of its kind holds.
// ---------------------------------------------------------------------------
template <int NT, bool GATED>
struct Small {
  static constexpr int NW = GATED ? 2 : 1;                        // weight tiles per step
  static constexpr int PER_SM = NT == 16 || (NT == 32 && !GATED) ? 2 : 1;
  static constexpr int S_MAX = NT == 16 && !GATED ? 8 : 4;
  static constexpr int DATA = NW * kWTile + NT * kRowBytes;       // a stage: [W | Up | X] codes
  static constexpr int SF = (NW + 1) * 2 * kAtom;                 // and scales
  static constexpr int STAGE = DATA + SF;
  // partials received: [source][W | Up][own token quad][128 rows][4 tokens]; the
  // owners' shares are whole quads, so S = 3 takes up to 3 ceil(NT / 12) of them,
  // S = 8 (NT = 16) 8
  static constexpr int QUADS = S_MAX == 8 ? 8 : 3 * ((NT / 4 + 2) / 3);
  static constexpr int RECV = NW * QUADS * 4 * kTile * 4;
  static constexpr int LIMIT = PER_SM == 2 ? 113 * 1024 : 227 * 1024;
  static constexpr int FIT = (LIMIT - 1024 - 256 - RECV) / STAGE;
  static constexpr int STAGES = FIT > 5 ? 5 : FIT;
  static constexpr int USED = 1024 + STAGES * STAGE + RECV + 256;
  static constexpr int SMEM = PER_SM == 2 ? (USED < 80 * 1024 ? 80 * 1024 : USED) : (USED < 120 * 1024 ? 120 * 1024 : USED);
  static constexpr uint32_t SF_COL = 128;                         // scales: 8 columns per operand and stage
  static constexpr uint32_t SF_STAGE = 8 * (NW + 1);
  static_assert(NT * NW <= 128 && SF_COL + STAGES * SF_STAGE <= 256, "TMEM columns");
  static_assert(STAGES >= 2 && SMEM <= LIMIT, "shared memory");
};

struct SmallParams {
  int64_t M, N, K;
  int steps, split, n_tiles;
  int last;                      // K = 64 products of the last step
  const uint16_t* x;             // XQ: bf16 rows, row stride ldx
  int64_t ldx;
  const uint8_t* sf[3];          // scales of W, Up, X
  int64_t sf_row;                // bytes per 128-row block of a scale buffer
  int64_t sf_bytes[3];
  void* y;
  int64_t ldy;
  bool pairs;                    // the rows of Y (fp32, bf16) take stores of column pairs
  uint8_t* q_codes;
  uint8_t* q_scales;
  unsigned* err;
};

// CNT tokens' outputs, one value per lane and token: rows t .. t + count - 1 of
// Y (count <= CNT), column n (the warp's 32 lanes hold 32 neighbouring columns,
// the first a multiple of 32).  The tokens go side by side through every step,
// so that their latencies overlap.
template <int OUT, int CNT>
__device__ __forceinline__ void store_lanes(const SmallParams& p, int64_t t, int64_t n, const float (&v)[CNT],
                                            int count) {
  static_assert(CNT % 2 == 0, "pairs of tokens");
  if (OUT == 1 && p.pairs) {
    // neighbouring lanes trade halves of two tokens, so that each stores two
    // columns of one of them (777 x 2048 x 1024: 6.4 -> 5.8 us)
    const int odd = threadIdx.x & 1;
    uint16_t* y = static_cast<uint16_t*>(p.y) + (t + odd) * p.ldy + (n - odd);
    const bool in = n < p.N;
#pragma unroll
    for (int i = 0; i < CNT; i += 2) {
      const uint32_t w = bf16x2(v[i], v[i + 1]);                // tokens t + i (low half), t + i + 1
      const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
      if (in && i + odd < count && NV_IDX(in_matrix(t + odd + i, n - odd, 2, p.M, p.N, p.ldy)))
        *reinterpret_cast<uint32_t*>(y) = odd ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
      y += 2 * p.ldy;
    }
  } else if (OUT == 0 && p.pairs) {
    const int odd = threadIdx.x & 1;
    float* y = static_cast<float*>(p.y) + (t + odd) * p.ldy + (n - odd);
    const bool in = n < p.N;
#pragma unroll
    for (int i = 0; i < CNT; i += 2) {
      const float o = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[i] : v[i + 1], 1);
      if (in && i + odd < count && NV_IDX(in_matrix(t + odd + i, n - odd, 2, p.M, p.N, p.ldy)))
        *reinterpret_cast<float2*>(y) = odd ? make_float2(o, v[i + 1]) : make_float2(v[i], o);
      y += 2 * p.ldy;
    }
  } else if constexpr (OUT < 2) {
    const bool in = n < p.N;
    uint8_t* y = static_cast<uint8_t*>(p.y) + (t * p.ldy + n) * (OUT == 0 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      if (in && i < count && NV_IDX(in_matrix(t + i, n, 1, p.M, p.N, p.ldy))) {
        if (OUT == 0) *reinterpret_cast<float*>(y) = v[i];
        else *reinterpret_cast<uint16_t*>(y) = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
      }
      y += p.ldy * (OUT == 0 ? 4 : 2);
    }
  } else {
    // 32 columns are a block of the next product's operand: N % 32 == 0, so it is
    // in or out as a whole (out: padding of the last atom, scale 0)
    static_assert(CNT <= 8, "a lane's codes are one word");
    const int lane = threadIdx.x & 31, l8 = lane & 7;
    const bool in = n - lane < p.N;
    uint32_t sb = 0;
    float q[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const uint32_t field = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[i]) & 0x7FFFFFFFu) >> 23;
      const bool bad = field == 255u;
      const uint32_t e = bad ? 255u : (field > 2u ? field - 2u : 0u);
      q[i] = bad ? 0.0f : __fmul_rn(v[i], __uint_as_float((254u - (bad ? 0u : e)) << 23));
      if (l8 == i) sb = e;
    }
    // lane c holds token i's code of column c in nibble i; transposed over each
    // eight lanes, lane i holds the eight columns of token i
    uint32_t w = e2m1x8(q);
#pragma unroll
    for (int d = 4; d >= 1; d /= 2) {
      const uint32_t low = d == 4 ? 0x0000FFFFu : d == 2 ? 0x00FF00FFu : 0x0F0F0F0Fu;
      const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, d);
      w = (lane & d) == 0 ? (w & low) | ((o & low) << (4 * d)) : (w & ~low) | ((o & ~low) >> (4 * d));
    }
    if (l8 < count && l8 < CNT) {
      const int64_t r = t + l8;
      if (in && NV_IDX(in_matrix(r, (n - l8) / 2, 4, p.M, p.N / 2, p.N / 2)))
        *reinterpret_cast<uint32_t*>(p.q_codes + r * (p.N / 2) + (n - l8) / 2) = w;
      const int64_t s = tiled_at(r, (n - lane) / 128, (p.N + 127) / 128, static_cast<int>((n - lane) / 32 % 4));
      if (lane < 8 && NV_IDX(s < scale_extent(p.M, p.N, 1, 32))) p.q_scales[s] = static_cast<uint8_t>(in ? sb : 0u);
    }
  }
}

// The quantized form of x[row][col .. col + 31] (zeros outside [M, K]).
struct Block {
  uint4 v[4];
};
__device__ __forceinline__ void load_block(const SmallParams& p, int row, int64_t col, Block& b) {
  const bool in = row < p.M && col < p.K &&        // K % 32 == 0: a block is in or out
                  NV_IDX(in_matrix(row, col, 32, p.M, p.K, p.ldx));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    b.v[i] = in ? ld_nc_v4(p.x + row * p.ldx + col + 8 * i) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint32_t quantize_block(const Block& b, uint4& codes) {
  const uint32_t* w = &b.v[0].x;
  uint32_t m2 = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) m2 = __vmaxu2(m2, w[j] & 0x7FFF7FFFu);
  const uint32_t field = max(m2 & 0xFFFFu, m2 >> 16) >> 7;
  const bool bad = field == 255u;
  const uint32_t sb = bad ? 255u : (field > 2u ? field - 2u : 0u);
  const float inv = __uint_as_float((254u - (bad ? 0u : sb)) << 23);
  uint32_t c[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint64_t f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f2_mul(bf16x2_to_f2(w[4 * h + j]), f2_pack(inv, inv));
    c[h] = bad ? 0u : e2m1x8_f2(f);
  }
  codes = make_uint4(c[0], c[1], c[2], c[3]);
  return sb;
}

// ACT: the gated form's activation, or -1 for a plain product.
template <int NT, int ACT, int OUT, bool XQ>
__global__ void __launch_bounds__(kThreads)
mx4_small_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmU,
                 const __grid_constant__ CUtensorMap tmX, const SmallParams p) {
  constexpr bool GATED = ACT >= 0;
  using C = Small<NT, GATED>;
  constexpr int DATA = C::DATA;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sf_base = smem + C::STAGES * DATA;
  float* recv = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE + C::RECV);
  uint64_t* empty = full + C::STAGES;
  uint64_t* done = empty + C::STAGES;
  uint64_t* got = done + 1;                          // the partials of this CTA's tokens have arrived
  uint32_t* slot = reinterpret_cast<uint32_t*>(got + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split;
  const int sidx = static_cast<int>(blockIdx.x % static_cast<unsigned>(S));
  const int tile = static_cast<int>(blockIdx.x / static_cast<unsigned>(S));
  const int nt = tile % p.n_tiles, mt = tile / p.n_tiles;
  const int64_t t0 = static_cast<int64_t>(mt) * NT;            // first token
  const int k_lo = p.steps * sidx / S, k_hi = p.steps * (sidx + 1) / S;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], XQ ? 5 : 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(got, 4 * S);                           // one arrival per epilogue warp of the cluster
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<1>(slot, 256);
  fence_before();
  __syncthreads();
  fence_after();
  if (S > 1) cluster_arrive();                       // (waited for before the first remote access)
  const uint32_t tmem = *slot;
  const int atoms = static_cast<int>((p.K + 127) / 128);
  auto sf_n = [&](int k) { return (atoms - 2 * k >= 2 ? 2u : 1u) * kAtom; };
  auto load = [&](int k, int stage) {
    const uint32_t fb = smem_u32(&full[stage]), n = sf_n(k);
    uint8_t* st = smem + stage * DATA;
    uint8_t* sf = sf_base + stage * C::SF;
    const int64_t off = nt * p.sf_row + 2ll * k * kAtom;
    if (!NV_IDX(off + n <= p.sf_bytes[0] && (XQ || (t0 >> 7) * p.sf_row + 2ll * k * kAtom + n <= p.sf_bytes[2])))
      return false;
    mbar_arrive_expect_tx(&full[stage], C::NW * (kWTile + n) + (XQ ? 0 : NT * kRowBytes + n));
    tma_load_2d(smem_u32(st), &tmW, k * kRowBytes, nt * kTile, fb);
    if (GATED) tma_load_2d(smem_u32(st + kWTile), &tmU, k * kRowBytes, nt * kTile, fb);
    bulk_load(smem_u32(sf), p.sf[0] + off, n, fb);
    if (GATED) bulk_load(smem_u32(sf + 2 * kAtom), p.sf[1] + off, n, fb);
    if (!XQ) {
      tma_load_2d(smem_u32(st + C::NW * kWTile), &tmX, k * kRowBytes, static_cast<int>(t0), fb);
      bulk_load(smem_u32(sf + C::NW * 2 * kAtom), p.sf[2] + (t0 >> 7) * p.sf_row + 2ll * k * kAtom, n, fb);
    }
    return true;
  };
  // Before the previous kernel's end, a hint to bring the first steps' weights
  // into L2 (gated, cold: 11.5 -> 10.7 us; for more steps it delays them).  They
  // are not loaded here, even where the kernel before is the same call's
  // quantizer: another host thread may queue a kernel that writes them in between.
  if (warp == 0 && lane == 0) {
    for (int k = k_lo; k < k_hi && k < k_lo + 4; ++k) {
      prefetch_2d(&tmW, k * kRowBytes, nt * kTile);
      if (GATED) prefetch_2d(&tmU, k * kRowBytes, nt * kTile);
    }
  }
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_phase = 0;
      for (int k = k_lo; k < k_hi; ++k) {
        if (!mbar_wait(&empty[stage], phase ^ 1, p.err) || !load(k, stage)) break;
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
      }
      // every copy in flight lands before the CTA can exit
      for (int s = 0; s < C::STAGES; ++s)
        if (armed & (1u << s)) mbar_wait(&full[s], (armed_phase >> s) & 1u, p.err);
    }
  } else if (warp == 1) {
    const bool lead = elect_one();
    const uint64_t dw = desc_k(smem_u32(smem)), dx = desc_k(smem_u32(smem) + C::NW * kWTile);
    const uint64_t ds = desc_atom(smem_u32(sf_base));
    int stage = 0;
    uint32_t phase = 0;
    for (int k = k_lo; k < k_hi; ++k) {
      if (!mbar_wait(&full[stage], phase, p.err)) break;
      fence_after();
      if (lead) {
        const uint64_t at = static_cast<uint64_t>(stage * (DATA >> 4));
        const uint64_t sf = ds + static_cast<uint64_t>(stage * (C::SF >> 4));
        // (tokens 64..127 of a 128-row block: their scales are 2 columns on)
        const uint32_t sft = tmem + C::SF_COL + C::SF_STAGE * stage;
        const uint32_t sfx = sft + 8 * C::NW + (NT == 64 ? 2 * (mt & 1) : 0);
        // both halves of each operand's scales (the second one of a last odd
        // atom is never read)
#pragma unroll
        for (int o = 0; o <= C::NW; ++o)
#pragma unroll
          for (int h = 0; h < 2; ++h) copy_atom<1>(sft + 8 * o + 4 * h, sf + ((2 * o + h) * kAtom >> 4));
        const int n_mma = k + 1 < p.steps ? 4 : p.last;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= n_mma) break;
          const uint32_t id = idesc_mx4(kTile, NT, j & 1), acc = k > k_lo || j > 0 ? 1u : 0u;
          mma_mx4<1>(tmem, dw + at + 2 * j, dx + at + 2 * j, id, sft + 4 * (j >> 1), sfx + 4 * (j >> 1), acc);
          if (GATED)
            mma_mx4<1>(tmem + NT, dw + at + (kWTile >> 4) + 2 * j, dx + at + 2 * j, id, sft + 8 + 4 * (j >> 1),
                       sfx + 4 * (j >> 1), acc);
        }
        commit1(&empty[stage]);
      }
      __syncwarp();
      if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
    }
    if (lead) {
      commit1(done);
      mbar_wait(done, 0, p.err);
    }
    __syncwarp();
  } else if (warp < 6) {
    const int q = warp & 3;
    bool good = true;
    if constexpr (XQ) {
      // X's tile of each K step: block b of row r to the swizzled 16-byte piece
      // b ^ (r % 8) of its row, its scale to the atom's place; kAhead steps of
      // loads in flight
      constexpr int kPer = NT * 8 / 128, kAhead = 4 / kPer;
      const int t = threadIdx.x - 64;
      int stage = 0;
      uint32_t phase = 0;
      for (int k0 = k_lo; k0 < k_hi && good; k0 += kAhead) {
        Block blk[kAhead][kPer];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            load_block(p, k0 + a < k_hi ? (t + 128 * i) / 8 : NT, (k0 + a) * static_cast<int64_t>(kStepK) + 32 * (t & 7),
                       blk[a][i]);
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          if (k0 + a >= k_hi || !good) break;
          if (lane == 0) good = mbar_wait(&empty[stage], phase ^ 1, p.err);
          good = __shfl_sync(0xFFFFFFFFu, good, 0);
          uint8_t* xt = smem + stage * DATA + C::NW * kWTile;
          uint8_t* sf = sf_base + stage * C::SF + C::NW * 2 * kAtom;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int r = (t + 128 * i) / 8, b = t & 7;
            if (r >= p.M) break;                     // (rows behind the last token feed columns nobody reads)
            uint4 codes;
            const uint32_t sb = quantize_block(blk[a][i], codes);
            *reinterpret_cast<uint4*>(xt + r * kRowBytes + 16 * (b ^ (r & 7))) = codes;
            sf[(b >> 2) * kAtom + r * 16 + (b & 3)] = static_cast<uint8_t>(sb);      // r < 16
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[stage]);
          if (++stage == C::STAGES) { stage = 0; phase ^= 1; }
        }
      }
    }
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int64_t n = static_cast<int64_t>(nt) * kTile + 32 * q + lane;
    const int cols = static_cast<int>(p.M - t0 < NT ? p.M - t0 : NT);
    if (OUT == 2 && sidx == 0 && t0 + NT >= p.M && (p.M & 127) != 0) {
      // the scale rows behind the last token (128-row padding of this atom)
      const int64_t r = (p.M & ~127ll) + 32 * q + lane;
      const int64_t s = tiled_at(r, nt, (p.N + 127) / 128, 0);
      if (r >= p.M && NV_IDX(s + 4 <= scale_extent(p.M, p.N, 1, 32))) *reinterpret_cast<uint32_t*>(p.q_scales + s) = 0u;
    }
    if (lane == 0) good = mbar_wait(done, 0, p.err) && good;
    good = __shfl_sync(0xFFFFFFFFu, good, 0);
    fence_after();
    if (S > 1) cluster_wait();                       // every CTA of the cluster runs and has its barriers
    // token quads per CTA: own sidx .. own sidx + own - 1; where this lane's
    // partials go: CTA `to`, its slot `tl`
    const int quads = (cols + 3) / 4, own = (quads + S - 1) / S;
    const uint32_t mine = smem_u32(recv + (sidx * C::NW * own * kTile + 32 * q + lane) * 4);
    int to = 0, tl = 0;
    uint32_t at = S > 1 ? peer_u32(mine, 0) : 0u;
    // (eight tokens at a time: unrolled further, the code's way into the
    // instruction cache took longer than the stores)
#pragma unroll 1
    for (int c = 0; c < cols; c += 8) {
      float g[8], u[8];
      tmem_ld(trow + c, g);
      if (GATED) tmem_ld(trow + NT + c, u);
      tmem_ld_wait(g, u);
      if (S == 1) {
        if (GATED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = act_value(g[i], ACT) * u[i];
        }
        if (good) store_lanes<OUT>(p, t0 + c, n, g, cols - c);
      } else {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          if (c + i >= cols) break;
          st_cluster_f4(at, g[i], g[i + 1], g[i + 2], g[i + 3]);
          if (GATED) st_cluster_f4(at + own * kTile * 16, u[i], u[i + 1], u[i + 2], u[i + 3]);
          at += kTile * 16;
          if (++tl == own) {
            tl = 0;
            at = peer_u32(mine, static_cast<uint32_t>(++to < S ? to : 0));
          }
        }
      }
    }
    if (S > 1) {
      __syncwarp();
      if (lane < S && lane * own < quads) arrive_cluster(peer_u32(smem_u32(got), static_cast<uint32_t>(lane)));
      const int q0 = sidx * own, n_own = quads - q0 < own ? quads - q0 : own;
      if (n_own > 0) {
        // the partials of this CTA's tokens, summed in CTA order
        good = mbar_wait_cluster(got, 0, p.err) && good;
        if (good) {
          const float4* r = reinterpret_cast<const float4*>(recv) + 32 * q + lane;
          const int src = C::NW * own * kTile;       // float4s per source
#pragma unroll 1
          for (int t = 0; t < n_own; ++t, r += kTile) {
            float4 g = r[0], u = GATED ? r[own * kTile] : g;
            for (int s = 1; s < S; ++s) {
              const float4 a = r[s * src];
              g.x = __fadd_rn(g.x, a.x);
              g.y = __fadd_rn(g.y, a.y);
              g.z = __fadd_rn(g.z, a.z);
              g.w = __fadd_rn(g.w, a.w);
              if (GATED) {
                const float4 b = r[s * src + own * kTile];
                u.x = __fadd_rn(u.x, b.x);
                u.y = __fadd_rn(u.y, b.y);
                u.z = __fadd_rn(u.z, b.z);
                u.w = __fadd_rn(u.w, b.w);
              }
            }
            float v[4] = {g.x, g.y, g.z, g.w};
            if (GATED) {
              const float uv[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = act_value(v[i], ACT) * uv[i];
            }
            store_lanes<OUT>(p, t0 + 4 * (q0 + t), n, v, cols - 4 * (q0 + t));
          }
        }
      }
    }
    fence_before();
  }
  if (S > 1 && !(warp >= 2 && warp < 6)) cluster_wait();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_dealloc<1>(tmem, 256);
  }
}

template <int NT, int ACT, int OUT, bool XQ>
cudaError_t launch_small(const Mx4Gemm& g, cudaStream_t s) {
  constexpr bool GATED = ACT >= 0;
  using C = Small<NT, GATED>;
  static bool attr_done[kMaxAttrDevices] = {};
  cudaError_t e = set_max_smem(mx4_small_kernel<NT, ACT, OUT, XQ>, C::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  SmallParams p{};
  p.M = g.M;
  p.N = g.N;
  p.K = g.K;
  p.steps = static_cast<int>((g.K + kStepK - 1) / kStepK);
  p.last = static_cast<int>((g.K - (p.steps - 1ll) * kStepK + 63) / 64);
  p.x = g.x_bf16;
  p.ldx = g.ldx;
  p.sf_row = (g.K + 127) / 128 * kAtom;
  p.sf[0] = g.w.scales;
  p.sf[1] = g.up.scales;
  p.sf[2] = g.x.scales;
  p.sf_bytes[0] = p.sf_bytes[1] = scale_extent(g.N, g.K, 1, 32);
  p.sf_bytes[2] = scale_extent(g.M, g.K, 1, 32);
  p.y = g.y;
  p.ldy = g.ldy;
  p.pairs = (reinterpret_cast<uintptr_t>(g.y) & (OUT == 0 ? 7u : 3u)) == 0 && g.ldy % 2 == 0 && g.N % 2 == 0;
  p.q_codes = g.q_codes;
  p.q_scales = g.q_scales;
  p.err = g.err;
  CUtensorMap mw, mu, mx;
  const int64_t rb = g.K / 2;
  if (!map_bytes(&mw, g.w.codes, g.N, rb, rb, kTile)) return cudaErrorInvalidValue;
  mu = mx = mw;
  if (GATED && !map_bytes(&mu, g.up.codes, g.N, rb, rb, kTile)) return cudaErrorInvalidValue;
  if (!XQ && !map_bytes(&mx, g.x.codes, g.M, rb, rb, NT)) return cudaErrorInvalidValue;
  p.n_tiles = static_cast<int>((g.N + kTile - 1) / kTile);
  const int tiles = p.n_tiles * static_cast<int>((g.M + NT - 1) / NT);
  // split over K while the CTAs fit the SMs at once: from 8 K steps on in up to
  // 4, with 64 tokens in 2 or 3 only from 16, and from 32 on in up to 8 (us, whole
  // / split: one token, 4096 x 4096, in 4 6.6 / 4.4, in 8 4.8; 11008 -> 4096 cold,
  // in 4 8.2, in 8 6.6; 64 gated tokens, 2048 -> 1024 in 4 8.1 / 6.8, 256 x 2048
  // x 2048 in 2 8.3 / 9.3, 64 x 4096 x 4096 in 2 11.3 / 10.1)
  p.split = 1;
  for (int c = 2; c <= C::S_MAX; ++c)
    if (static_cast<int64_t>(tiles) * c <= C::PER_SM * sm_count() &&
        p.steps >= (c > 4 ? 32 : NT == 64 && c < 4 ? 16 : 8))
      p.split = c;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  e = launch_k(mx4_small_kernel<NT, ACT, OUT, XQ>, dim3(static_cast<unsigned>(tiles * p.split)), dim3(kThreads),
               C::SMEM, s, attr, 1, mw, mu, mx, p);
  return e;
}

template <int ACT, int OUT>
cudaError_t small(const Mx4Gemm& g, cudaStream_t s) {
  if (g.M <= 16) return launch_small<16, ACT, OUT, false>(g, s);
  return g.M <= 32 ? launch_small<32, ACT, OUT, false>(g, s) : launch_small<64, ACT, OUT, false>(g, s);
}
template <int ACT>
cudaError_t small_gated(const Mx4Gemm& g, cudaStream_t s) {
  if (g.y_dtype == 2) return small<ACT, 2>(g, s);
  return g.y_dtype == 0 ? small<ACT, 0>(g, s) : small<ACT, 1>(g, s);
}
cudaError_t small_any(const Mx4Gemm& g, cudaStream_t s) {
  if (g.up.codes == nullptr) return g.y_dtype == 0 ? small<-1, 0>(g, s) : small<-1, 1>(g, s);
  return g.act == kActSilu ? small_gated<kActSilu>(g, s) : small_gated<kActGeluTanh>(g, s);
}

}  // namespace

// Up to 8 tokens.  Measured (us a call, cold weights, quantizing in the product /
// in a launch of its own): 4096 -> 11008 4 tokens 8.0 / 9.2, 8 8.7 / 8.8, 12 9.3 /
// 8.9, 16 10.0 / 9.5; 11008 -> 4096 4 8.0 / 9.4, 8 8.7 / 9.5, 16 10.0 / 9.7; 4096
// -> 4096 8 5.9 / 6.8, 16 6.9 / 6.9; 2048 -> 1024 8 4.3 / 6.2.
bool mx4_takes_bf16(int64_t M) { return M <= 8; }

// Up to 32 tokens; while the tiles of 64 tokens x 128 weight rows fit the SMs at
// once, also a plain product of more, and a gated one up to 128.  Measured (us,
// this kernel / the pair's):
//   plain   333 x 1504 x 1001 fp32 5.1 / 12.1, 1024 x 2048 x 1024 bf16 5.9 / 7.6,
//           512 x 4096 x 2048 bf16 8.4 / 10.1; at more tiles than SMs,
//           256 x 1024 x 6144, 9.8 / 6.3
//   gated   32 x 4096 x 11008 10.1 / 17.6, 64 x 2048 x 1024 6.8 / 8.1, 128 x 2048 x
//           1024 7.1 / 8.2, 512 x 2048 x 1024 8.3 / 8.3, 777 x 2048 x 1024 8.6 / 8.4
bool small_pays(const Mx4Gemm& g) {
  if (g.M <= 32) return true;
  const bool one_wave = (g.M + 63) / 64 * ((g.N + kTile - 1) / kTile) <= sm_count();
  return one_wave && (g.up.codes == nullptr || g.M <= 128);
}

cudaError_t launch_mx4_gemm(const Mx4Gemm& g, cudaStream_t s) {
  if (g.x_bf16 != nullptr)
    return g.y_dtype == 0 ? launch_small<16, -1, 0, true>(g, s) : launch_small<16, -1, 1, true>(g, s);
  return small_pays(g) ? small_any(g, s) : launch_mx4_pair(g, s);
}

NV_DEFINE_BOUNDS_READER(bounds_flags_mx4_gemm)

}  // namespace nvfp4

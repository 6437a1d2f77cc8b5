// MXFP4 products of many rows on CTA pairs (tcgen05 cta_group::2): see
// mx4_gemm.cu for the operators and the kernel for few rows.
//
// A pair computes a 256 x 256 accumulator tile; each CTA loads its own 128
// rows of A and of B per K step of 256 (16 KB each, 128-byte swizzle) and the
// block scales of its A rows and of all 256 B rows.  Gated: CTA 0's B rows are
// 128 gate rows and CTA 1's the up rows of the same outputs, so a tile is
// 256 x 128 outputs with G in columns 0..127 and U in columns 128..255.
//
// TMEM (512 columns): two accumulators that share 96 columns (0..255 and
// 160..415), and four slots of block scales (24 columns each).  The epilogue of
// a tile first takes the shared 96 columns into registers and lets the next
// tile's MMAs start; the rest is drained under them.  (Two slots, whose copies
// run at most two steps ahead, cost 3 %.)
//
// Measured (us, burst / loop of 1.5 s at the 1000 W cap): 32768 x 4096 x 4096 219 /
// 249 (5.0 / 4.4 PFLOP/s), 8192 x 11008 x 4096 135 / 149, gated 8192 x 4096 x 11008
// 285 / 316.  In the loop the SM clock is 1.5 to 1.6 GHz, and this 60 to 68 % of the
// tensor peak at that clock.  Power and operand supply bound it together: in a
// burst 5.5 PFLOP/s became 6.0 without the scale copies, 7.4 without the loads.
//
// Warps: 0 loads, 1 MMA issue (leader CTA), 2..9 epilogue (two per TMEM lane
// quadrant, each half of the columns: with four warps the epilogue of a lone
// 256 x 256 x 256 tile took 1 us more, 2 us gated), 10 scale copies (leader
// CTA; its own thread, so that the copies do not queue behind MMAs).
#include "mx4_common.cuh"

namespace nvfp4 {
namespace {

using namespace umma;

constexpr int kThreads = 352;
constexpr int kOperand = 128 * kRowBytes;                  // 16 KB
constexpr int kSfA = 2 * kAtom, kSfB = 4 * kAtom;          // scales of a K step: 128 rows of A, 256 of B
constexpr int kStage = 2 * kOperand + kSfA + kSfB;
constexpr int kStages = 5;
constexpr uint32_t kAcc1 = 160, kShared = 96, kSlotCol = 416, kSlot = 24, kSlots = 4;
static_assert(kAcc1 + kShared == 256 && kAcc1 + 256 == kSlotCol && kSlotCol + kSlots * kSlot == 512, "TMEM columns");

template <int OUT>
struct Pair {
  // epilogue staging per warp: 32 rows of 32 fp32 or 64 bf16 outputs, or the
  // codes of 64, padded by 16 bytes (bank conflicts)
  static constexpr int COLS = OUT == 0 ? 32 : 64;
  static constexpr int STRIDE = (OUT == 2 ? 32 : 128) + 16;
  static constexpr int WARP = 32 * STRIDE;
  static constexpr int SMEM = 1024 + kStages * kStage + 8 * WARP + 256;
  static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
};

struct PairParams {
  int64_t M, N, K;
  int row_tiles, col_tiles, steps;
  int last;                      // K = 64 products of the last step
  void* y;
  int64_t ldy;
  bool vec;                      // y rows can take 16-byte stores
  uint8_t* q_codes;
  uint8_t* q_scales;
  unsigned* err;
};

// 32 staged rows of 128 bytes to memory: 16-byte pieces where the rows allow
// them, single elements otherwise (and at the end of a row).
template <int OUT>
__device__ __forceinline__ void store_rows(const PairParams& p, const uint8_t* stg, int64_t row0, int64_t col0,
                                           int lane) {
  constexpr int SIZE = OUT == 0 ? 4 : 2, PER = 16 / SIZE, COLS = Pair<OUT>::COLS;
  uint8_t* y = static_cast<uint8_t*>(p.y);
  if (p.vec && col0 + COLS <= p.N) {
    const int64_t col = col0 + PER * (lane & 7);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      if (row0 + r < p.M && NV_IDX(in_matrix(row0 + r, col, PER, p.M, p.N, p.ldy)))
        *reinterpret_cast<uint4*>(y + ((row0 + r) * p.ldy + col) * SIZE) =
            *reinterpret_cast<const uint4*>(stg + r * Pair<OUT>::STRIDE + 16 * (lane & 7));
    }
  } else {
#pragma unroll 8
    for (int i = 0; i < COLS; ++i) {
      const int r = OUT == 0 ? i : i >> 1, c = OUT == 0 ? lane : (i & 1) * 32 + lane;
      if (row0 + r < p.M && col0 + c < p.N && NV_IDX(in_matrix(row0 + r, col0 + c, 1, p.M, p.N, p.ldy))) {
        if (OUT == 0)
          reinterpret_cast<uint32_t*>(y)[(row0 + r) * p.ldy + col0 + c] =
              *reinterpret_cast<const uint32_t*>(stg + r * Pair<OUT>::STRIDE + 4 * c);
        else
          reinterpret_cast<uint16_t*>(y)[(row0 + r) * p.ldy + col0 + c] =
              *reinterpret_cast<const uint16_t*>(stg + r * Pair<OUT>::STRIDE + 2 * c);
      }
    }
  }
}

// 32 outputs of this lane's row into its staging row, at output column `at`.
template <int OUT>
__device__ __forceinline__ void stage32(uint8_t* stg_row, int at, const float (&v)[32]) {
  if (OUT == 0) {
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      *reinterpret_cast<float4*>(stg_row + (at + i) * 4) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
      *reinterpret_cast<uint4*>(stg_row + (at + i) * 2) =
          make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]), bf16x2(v[i + 4], v[i + 5]),
                     bf16x2(v[i + 6], v[i + 7]));
  }
}

// One 32-column block of this lane's row to MXFP4: 16 bytes of codes, the
// scale byte returned.
__device__ __forceinline__ uint32_t quantize32(const float (&v)[32], uint8_t* dst) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const uint32_t field = m >> 23;
  const bool bad = field == 255u;
  const uint32_t sb = bad ? 255u : (field > 2u ? field - 2u : 0u);
  const float inv = __uint_as_float((254u - (bad ? 0u : sb)) << 23);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __fmul_rn(v[8 * j + i], inv);
    w[j] = bad ? 0u : e2m1x8(t);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  return sb;
}

// 32 outputs at column col0 + 32 e of the warp's 64 (e 0, then 1): staged, and
// stored when the staging rows are full.
template <int OUT>
__device__ __forceinline__ void put32(const PairParams& p, uint8_t* stg, int lane, int64_t row0, int64_t col0, int e,
                                      const float (&v)[32]) {
  stage32<OUT>(stg + lane * Pair<OUT>::STRIDE, OUT == 0 ? 0 : 32 * e, v);
  if (OUT == 0 || e == 1) {
    __syncwarp();
    store_rows<OUT>(p, stg, row0, OUT == 0 ? col0 + 32 * e : col0, lane);
    __syncwarp();
  }
}

// The epilogue of one tile by one warp: 32 rows, and of the accumulator's eight
// 32-column blocks (gated: of its four pairs G, U) the blocks 0 1 4 5 of half
// 0 or 2 3 6 7 of half 1 (pairs 0 1 or 2 3).  The other accumulator shares the
// blocks 5..7 of accumulator 0 and 0..2 of accumulator 1, so of a half's
// blocks 4 h + 2 half + {0, 1} (h = 1 or 0; of its pairs' U or G) both or one:
// `held`.  These are taken into registers first, and `release` then lets the
// next tile's MMAs start.  Accumulator and half are run-time values: four
// copies of this code did not fit the instruction cache (8192 x 1024 x 2048
// gated: 44 us).
template <int ACT, int OUT, class Release>
__device__ __forceinline__ void drain(const PairParams& p, uint32_t trow, uint8_t* stg, int64_t row0, int ct, int lane,
                                      uint32_t buf, int half, Release release) {
  constexpr bool GATED = ACT >= 0;
  const uint32_t acc = trow + (buf ? kAcc1 : 0u);
  const bool held[2] = {buf == 1 || half == 1, buf == 0 || half == 0};
  // first the held blocks: gated, U (accumulator 0) or G of pairs 2 half + e
  const uint32_t first = acc + 32 * (buf ? 0 : 4) + 64 * half;
  float hold[2][32];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (held[e]) tmem_ld(first + 32 * e, hold[e]);
#pragma unroll
  for (int e = 0; e < 2; ++e) tmem_ld_wait(hold[e]);
  fence_before();
  __syncwarp();
  release();
  if constexpr (GATED) {
    const uint32_t second = acc + 32 * (buf ? 4 : 0) + 64 * half;
    const int64_t col0 = static_cast<int64_t>(ct) * 128 + 64 * half;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float o[32];
      if (!held[e]) tmem_ld(first + 32 * e, hold[e]);
      tmem_ld(second + 32 * e, o);
      tmem_ld_wait(hold[e], o);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float g = buf ? hold[e][j] : o[j], u = buf ? o[j] : hold[e][j];
        o[j] = act_value(g, ACT) * u;
      }
      if constexpr (OUT == 2) {
        const uint32_t sb = quantize32(o, stg + lane * Pair<OUT>::STRIDE + 16 * e);
        word |= (col0 + 32 * e < p.N ? sb : 0u) << (8 * e);
      } else {
        put32<OUT>(p, stg, lane, row0, col0, e, o);
      }
    }
    if constexpr (OUT == 2) {
      __syncwarp();
      // codes: 32 bytes per row, 2 lanes a row; a lane's 16 bytes are one block
      const int64_t col = col0 + 32 * (lane & 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * i + (lane >> 1);
        if (row0 + r < p.M && col < p.N && NV_IDX(in_matrix(row0 + r, col / 2, 16, p.M, p.N / 2, p.N / 2)))
          *reinterpret_cast<uint4*>(p.q_codes + (row0 + r) * (p.N / 2) + col / 2) =
              *reinterpret_cast<const uint4*>(stg + r * Pair<OUT>::STRIDE + 16 * (lane & 1));
      }
      // scales: this tile is one atom wide, the warp's two blocks half of a
      // row's word; the rows behind the last one up to the padding's end get zeros
      const int64_t row = row0 + lane;
      const int64_t s = tiled_at(row, ct, (p.N + 127) / 128, 2 * half);
      if (row < (p.M + 127) / 128 * 128 && NV_IDX(s + 2 <= scale_extent(p.M, p.N, 1, 32)))
        *reinterpret_cast<uint16_t*>(p.q_scales + s) = static_cast<uint16_t>(row < p.M ? word : 0u);
      __syncwarp();
    }
  } else {
    // the pair of blocks with the held ones, then the other pair
#pragma unroll 1
    for (int g = 0; g < 2; ++g) {
      const int h = g == 0 ? (buf ? 0 : 1) : (buf ? 1 : 0);
      const uint32_t at = acc + 128 * h + 64 * half;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (g == 1 || !held[e]) tmem_ld(at + 32 * e, hold[e]);
      tmem_ld_wait(hold[0], hold[1]);
      const int64_t col0 = static_cast<int64_t>(ct) * 256 + 128 * h + 64 * half;
#pragma unroll
      for (int e = 0; e < 2; ++e) put32<OUT>(p, stg, lane, row0, col0, e, hold[e]);
    }
  }
}

// ACT: the gated form's activation, or -1 for a plain product.
template <int ACT, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
mx4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmSA,
                const __grid_constant__ CUtensorMap tmSB0, const __grid_constant__ CUtensorMap tmSB1,
                const PairParams p) {
  constexpr bool GATED = ACT >= 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sf = smem + kStages * 2 * kOperand;               // [stages][A atoms | B atoms]
  uint8_t* stg = smem + kStages * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + 8 * Pair<OUT>::WARP);
  uint64_t* empty = full + kStages;
  uint64_t* sf_full = empty + kStages;                       // [kSlots] the slot's scales are in TMEM
  uint64_t* acc_full = sf_full + kSlots;                     // [2]
  uint64_t* acc_free = acc_full + 2;                         // the shared columns of the last tile are taken
  uint64_t* done = acc_free + 1;                             // [2]
  uint32_t* slot_word = reinterpret_cast<uint32_t*>(done + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (uint32_t s = 0; s < kSlots; ++s) mbar_init(&sf_full[s], 1);
    mbar_init(&acc_full[0], 1);
    mbar_init(&acc_full[1], 1);
    mbar_init(acc_free, 16);                                 // one arrival per epilogue warp of both CTAs
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster_sync();
  if (warp == 1) tmem_alloc<2>(slot_word, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *slot_word;
  const int total = p.row_tiles * p.col_tiles;
  // this CTA's loads of a K step: B and its scales, A and its scales
  auto load = [&](int rt, int ct, int k, int stage) {
    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kStage);
    const uint32_t bar = peer_u32(smem_u32(&full[stage]), 0);
    const uint32_t a = smem_u32(smem + stage * 2 * kOperand), b = a + kOperand;
    const uint32_t sa = smem_u32(sf + stage * (kSfA + kSfB)), s = sa + kSfA;
    load_2d_pair(b, GATED && rank ? &tmB1 : &tmB0, k * kRowBytes, (GATED ? ct : 2 * ct + static_cast<int>(rank)) * 128,
                 bar);
    load_2d_pair(s, &tmSB0, k * kSfA / 8, GATED ? ct : 2 * ct, bar);
    load_2d_pair(s + kSfA, GATED ? &tmSB1 : &tmSB0, k * kSfA / 8, GATED ? ct : 2 * ct + 1, bar);
    const int block = 2 * rt + static_cast<int>(rank);       // 128-row block
    load_2d_pair(a, &tmA, k * kRowBytes, block * 128, bar);
    load_2d_pair(sa, &tmSA, k * kSfA / 8, block, bar);
  };
  // before the previous kernel's end: a hint to bring the first steps' weights
  // into L2 (no load, which could meet a write queued by another host thread)
  if (warp == 0 && lane == 0 && pair < total) {
    int rt, ct;
    tile_at(pair, p.row_tiles, p.col_tiles, rt, ct);
    for (int k = 0; k < kStages && k < p.steps; ++k)
      prefetch_2d(GATED && rank ? &tmB1 : &tmB0, k * kRowBytes, (GATED ? ct : 2 * ct + static_cast<int>(rank)) * 128);
  }
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_phase = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        int rt, ct;
        tile_at(tile, p.row_tiles, p.col_tiles, rt, ct);
        for (int k = 0; k < p.steps; ++k) {
          if (!mbar_wait(&empty[stage], phase ^ 1, p.err)) { ok = false; break; }
          load(rt, ct, k, stage);
          armed |= 1u << stage;
          armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      // this CTA's copies land before it can exit
      for (int s = 0; s < kStages; ++s)
        if (armed & (1u << s)) mbar_wait(rank == 0 ? &full[s] : &empty[s], (armed_phase >> s) & 1u, p.err);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const bool lead = elect_one();
      const uint64_t da = desc_k(smem_u32(smem)), db = desc_k(smem_u32(smem) + kOperand);
      int stage = 0;
      uint32_t phase = 0, slot = 0, slot_phase = 0, free_phase = 0, buf = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        // the epilogue has the shared columns of the previous tile (and, being
        // in order, all of the tile before)
        if (!mbar_wait(acc_free, free_phase ^ 1, p.err)) break;
        free_phase ^= 1;
        fence_after();
        const uint32_t d = tmem + (buf ? kAcc1 : 0u);
        for (int k = 0; k < p.steps; ++k) {
          if (!mbar_wait(&full[stage], phase, p.err) || !mbar_wait(&sf_full[slot], slot_phase, p.err)) {
            ok = false;
            break;
          }
          fence_after();
          if (lead) {
            const uint64_t at = static_cast<uint64_t>(stage * (2 * kOperand >> 4));
            const uint32_t sfa = tmem + kSlotCol + kSlot * slot, sfb = sfa + 8;
            if (k + 1 < p.steps || p.last == 4) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_mx4<2>(d, da + at + 2 * j, db + at + 2 * j, idesc_mx4(256, 256, j & 1), sfa + 4 * (j >> 1),
                           sfb + 8 * (j >> 1), k > 0 || j > 0 ? 1u : 0u);
            } else {
              for (int j = 0; j < p.last; ++j)
                mma_mx4<2>(d, da + at + 2 * j, db + at + 2 * j, idesc_mx4(256, 256, j & 1), sfa + 4 * (j >> 1),
                           sfb + 8 * (j >> 1), k > 0 || j > 0 ? 1u : 0u);
            }
            commit2_both(&empty[stage]);
          }
          __syncwarp();
          if (++stage == kStages) { stage = 0; phase ^= 1; }
          if (++slot == kSlots) { slot = 0; slot_phase ^= 1; }
        }
        if (lead) commit2_both(&acc_full[buf]);
        __syncwarp();
        buf ^= 1;
      }
      // the peer's last arrivals here have landed (see cluster_sync)
      mbar_wait(acc_free, free_phase ^ 1, p.err);
      if (lead) {
        commit2_lead(&done[0]);
        mbar_wait(&done[0], 0, p.err);
      }
      __syncwarp();
    }
  } else if (warp == 10) {
    if (rank == 0) {
      const bool lead = elect_one();
      const uint64_t ds = desc_atom(smem_u32(sf));
      int stage = 0, old = 0;                                // old: the stage of the step kSlots back
      uint32_t phase = 0, slot = 0, old_phase = 0, n = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        for (int k = 0; k < p.steps; ++k) {
          // the slot's last reader was the step kSlots back: its stage's `empty`
          // (which cannot complete again before this step's scales are there)
          if (!mbar_wait(&full[stage], phase, p.err) || (n >= kSlots && !mbar_wait(&empty[old], old_phase, p.err))) {
            ok = false;
            break;
          }
          fence_after();
          if (lead) {
            const uint64_t s = ds + static_cast<uint64_t>(stage * ((kSfA + kSfB) >> 4));
            const uint32_t sfa = tmem + kSlotCol + kSlot * slot, sfb = sfa + 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              copy_atom<2>(sfa + 4 * h, s + h * (kAtom >> 4));
              copy_atom<2>(sfb + 8 * h, s + ((kSfA + h * kAtom) >> 4));
              copy_atom<2>(sfb + 8 * h + 4, s + ((2 * kSfA + h * kAtom) >> 4));
            }
            commit2_lead(&sf_full[slot]);
          }
          __syncwarp();
          if (n >= kSlots) {
            if (++old == kStages) { old = 0; old_phase ^= 1; }
          } else {
            ++n;
          }
          if (++stage == kStages) { stage = 0; phase ^= 1; }
          if (++slot == kSlots) slot = 0;
        }
      }
      if (lead) {
        commit2_lead(&done[1]);
        mbar_wait(&done[1], 0, p.err);
      }
      __syncwarp();
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * q) << 16);
    uint8_t* mine = stg + (warp - 2) * Pair<OUT>::WARP;
    const uint32_t free_bar = peer_u32(smem_u32(acc_free), 0);
    uint32_t buf = 0, acc_phase = 0;
    auto release = [&]() {
      if (lane == 0) arrive_cluster(free_bar);
    };
    for (int tile = pair; tile < total; tile += npairs) {
      int rt, ct;
      tile_at(tile, p.row_tiles, p.col_tiles, rt, ct);
      bool ok = true;
      if (lane == 0) ok = mbar_wait(&acc_full[buf], acc_phase, p.err);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      fence_after();
      const int64_t row0 = static_cast<int64_t>(rt) * 256 + rank * 128 + 32 * q;
      drain<ACT, OUT>(p, trow, mine, row0, ct, lane, buf, half, release);
      acc_phase ^= buf;                                      // both accumulators used once per phase
      buf ^= 1;
    }
  }
  fence_before();
  __syncthreads();
  cluster_sync();                                        // neither CTA leaves while its peer may still signal it
  if (warp == 1) {
    fence_after();
    tmem_dealloc<2>(tmem, 512);
  }
}

// The scale buffer as int64 [128-row blocks][atoms * 64], boxes of two atoms.
bool map_scales(CUtensorMap* tm, const uint8_t* scales, int64_t rows, int64_t K) {
  const int64_t atoms = (K + 127) / 128;
  return map_2d(tm, CU_TENSOR_MAP_DATA_TYPE_INT64, scales, (rows + 127) / 128, atoms * (kAtom / 8), atoms * kAtom, 1,
                2 * kAtom / 8, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int ACT, int OUT>
cudaError_t launch(const Mx4Gemm& g, cudaStream_t s) {
  constexpr bool GATED = ACT >= 0;
  static bool attr_done[kMaxAttrDevices] = {};
  cudaError_t e = set_max_smem(mx4_pair_kernel<ACT, OUT>, Pair<OUT>::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  PairParams p{};
  p.M = g.M;
  p.N = g.N;
  p.K = g.K;
  p.row_tiles = static_cast<int>((g.M + 255) / 256);
  p.col_tiles = static_cast<int>((g.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256));
  p.steps = static_cast<int>((g.K + kStepK - 1) / kStepK);
  p.last = static_cast<int>((g.K - (p.steps - 1ll) * kStepK + 63) / 64);
  p.y = g.y;
  p.ldy = g.ldy;
  p.vec = (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0 && g.ldy % (OUT == 0 ? 4 : 8) == 0;
  p.q_codes = g.q_codes;
  p.q_scales = g.q_scales;
  p.err = g.err;
  const int64_t rb = g.K / 2, tiles = static_cast<int64_t>(p.row_tiles) * p.col_tiles;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const Mx4Operand& up = GATED ? g.up : g.w;
  CUtensorMap a, b0, b1, sa, sb0, sb1;
  if (!map_bytes(&a, g.x.codes, g.M, rb, rb, 128) || !map_bytes(&b0, g.w.codes, g.N, rb, rb, 128) ||
      !map_bytes(&b1, up.codes, g.N, rb, rb, 128) || !map_scales(&sa, g.x.scales, g.M, g.K) ||
      !map_scales(&sb0, g.w.scales, g.N, g.K) || !map_scales(&sb1, up.scales, g.N, g.K))
    return cudaErrorInvalidValue;
  const int64_t pairs = tiles < sm_count() / 2 ? tiles : sm_count() / 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  e = launch_k(mx4_pair_kernel<ACT, OUT>, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads), Pair<OUT>::SMEM, s,
               attr, 1, a, b0, b1, sa, sb0, sb1, p);
  return e;
}

template <int ACT>
cudaError_t launch_act(const Mx4Gemm& g, cudaStream_t s) {
  if (g.y_dtype == 2) return launch<ACT, 2>(g, s);
  return g.y_dtype == 0 ? launch<ACT, 0>(g, s) : launch<ACT, 1>(g, s);
}

}  // namespace

cudaError_t launch_mx4_pair(const Mx4Gemm& g, cudaStream_t s) {
  if (g.up.codes == nullptr) return g.y_dtype == 0 ? launch<-1, 0>(g, s) : launch<-1, 1>(g, s);
  return g.act == kActSilu ? launch_act<kActSilu>(g, s) : launch_act<kActGeluTanh>(g, s);
}

NV_DEFINE_BOUNDS_READER(bounds_flags_mx4_pair)

}  // namespace nvfp4

// The trainer's gated projection in bf16 and its backward pass, on the
// 5th-generation tensor cores (tcgen05 kind::f16, fp32 accumulators in TMEM):
//
//     H  = act(G) * U,        G = X Wg^T, U = X Wu^T          (one kernel)
//     dG = dH U act'(G),      dU = dH act(G)                  (element-wise)
//     dX = dG Wg + dU Wu                                      (one kernel)
//     dWg = dG^T X,           dWu = dU^T X                    (one kernel)
//
// G and U stay fp32 from the accumulators to the element-wise backward (kept
// in the forward pass, or computed again): rounding them to bf16 there would
// add an error of the size of the gradients' own rounding twice over.  dG and
// dU are rounded to bf16 once, because the tensor cores take them so.
#include "act.cuh"
#include "umma.cuh"

namespace nvfp4 {
namespace {

using namespace umma;

// ---------------------------------------------------------------------------
// The product kernel: CTA pairs (cta_group::2), 256 x 256 accumulator tiles,
// persistent over the tiles.  Per K step of 64 each CTA loads its 128 rows of
// A and its 128 columns of B (16 KB each, 128-byte swizzle) into a six-stage
// ring; the leader issues four MMAs of 256 x 256 x 16.  Two accumulators (all
// 512 TMEM columns): the epilogue of one tile runs under the MMAs of the next.
//
//   kForward  A = X, B = [Wg rows | Wu rows] (CTA 0 loads the 128 gate rows,
//             CTA 1 the up rows of the same outputs): a tile is 256 x 128 of H
//             with G and U of one output in columns c and 128 + c.
//   kGradX    two K segments, dG Wg then dU Wu; W is read along its rows, so B
//             is MN-major.
//   kGradW    A = dG or dU read along its rows (MN-major), B = X likewise; the
//             reduction runs over the tokens.
//
// Bound by the tensor pipe in a single launch (97 % active in the gradients, 91 %
// in the forward pass that also writes 8 bytes of projections per output), by the
// power cap in a long run.  8192 x 4096 x 11008 (us, burst / loop of 1.5 s): forward
// 930 / 1035 (1.59 / 1.43 PFLOP/s), with the projections kept 1014 / 1140, dX 944 /
// 1102, dW 949 / 1117; a cuBLAS product of that size 911 / 1065.  Up to 256 tokens
// dX has few tiles of a long reduction, which nothing splits: 104 us with the slopes
// for one token, where reading the weights takes 28.
// ---------------------------------------------------------------------------
enum Mode { kForward, kGradX, kGradW };

constexpr int kStages = 6;
constexpr int kHalf = 128 * kRowBytes;             // 16 KB: one CTA's operand tile of a K step
constexpr int kStage = 2 * kHalf;
constexpr int kStgStride = 64 * 2 + 16;            // staging row: 64 bf16, padded by 16 bytes (bank conflicts)
constexpr int kStgWarp = 32 * kStgStride;
constexpr int kSmem = 1024 + kStages * kStage + 4 * kStgWarp + 256;
constexpr int kThreads = 192;                      // warps: 0 loads, 1 MMA, 2..5 epilogue
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");

struct Params {
  int64_t rows, cols;          // of the output: H [M, F], dX [M, K], dW [F, K]
  int row_tiles, col_tiles;    // 256-row tiles; 128 (forward) or 256 columns
  int steps, segments;         // K steps of 64 per segment
  int mats;                    // kGradW: matrices (1 or 2)
  int act;
  uint16_t* out[2];
  int64_t ldo;
  float* saved;                // kForward: G and U, or null
  int64_t sv_rb, sv_cb;        // its 32 x 32 blocks per column / row
  unsigned* err;
};

// bf16 x bf16 -> fp32, M = N = 256 over the pair; bits 15 / 16: A / B MN-major.
template <Mode MODE>
__device__ __forceinline__ constexpr uint32_t idesc() {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((MODE == kGradW ? 1u : 0u) << 15) |
         ((MODE == kForward ? 0u : 1u) << 16) | (uint32_t(256 >> 3) << 17) | (uint32_t(256 >> 4) << 24);
}

// Saved projections: 32 x 32 blocks [row block][column block], each as
// [8 column quads][32 rows][4] fp32, so that the lane that holds a row writes
// and reads 16 bytes next to its neighbours'; U behind G.
__device__ __forceinline__ int64_t saved_at(int64_t rb, int64_t cb, int64_t n_cb) { return (rb * n_cb + cb) * 1024; }

template <Mode MODE>
__global__ void __launch_bounds__(kThreads, 1)
gated_pair_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                  const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                  const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* stg = smem + kStages * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + 4 * kStgWarp);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;            // [2]
  uint64_t* acc_empty = acc_full + 2;              // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);                 // one arrival per epilogue warp of both CTAs
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster_sync();
  if (warp == 1) tmem_alloc<2>(slot, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *slot;
  const int per_mat = p.row_tiles * p.col_tiles;
  const int total = per_mat * p.mats;
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_phase = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        const int mat = tile / per_mat;
        int r, c;
        tile_at(tile - mat * per_mat, p.row_tiles, p.col_tiles, r, c);
        const int row = r * 256 + static_cast<int>(rank) * 128;
        const int col = MODE == kForward ? c * 128 : c * 256 + static_cast<int>(rank) * 128;
        for (int seg = 0; seg < p.segments && ok; ++seg) {
          const CUtensorMap* ta = (MODE == kGradW ? mat : seg) ? &tmA1 : &tmA0;
          const CUtensorMap* tb = (MODE == kForward ? static_cast<int>(rank) : seg) ? &tmB1 : &tmB0;
          for (int k = 0; k < p.steps; ++k) {
            if (!mbar_wait(&empty[stage], phase ^ 1, p.err)) { ok = false; break; }
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kStage);
            const uint32_t bar = peer_u32(smem_u32(&full[stage]), 0);
            const uint32_t a = smem_u32(smem + stage * kStage), b = a + kHalf;
            if (MODE == kGradW) {                  // 64 tokens x 2 x 64 outputs
              load_2d_pair(a, ta, row * 2, k * 64, bar);
              load_2d_pair(a + kHalf / 2, ta, row * 2 + kRowBytes, k * 64, bar);
            } else {
              load_2d_pair(a, ta, k * kRowBytes, row, bar);
            }
            if (MODE == kForward) {
              load_2d_pair(b, tb, k * kRowBytes, col, bar);
            } else {
              load_2d_pair(b, tb, col * 2, k * 64, bar);
              load_2d_pair(b + kHalf / 2, tb, col * 2 + kRowBytes, k * 64, bar);
            }
            armed |= 1u << stage;
            armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == kStages) { stage = 0; phase ^= 1; }
          }
        }
      }
      // this CTA's copies land before it can exit
      for (int s = 0; s < kStages; ++s)
        if (armed & (1u << s)) mbar_wait(rank == 0 ? &full[s] : &empty[s], (armed_phase >> s) & 1u, p.err);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const bool lead = elect_one();
      const uint64_t da = MODE == kGradW ? desc_mn(smem_u32(smem), kHalf / 2) : desc_k(smem_u32(smem));
      const uint64_t db = MODE == kForward ? desc_k(smem_u32(smem) + kHalf) : desc_mn(smem_u32(smem) + kHalf, kHalf / 2);
      constexpr uint64_t kStepA = (MODE == kGradW ? 2048 : 32) >> 4, kStepB = (MODE == kForward ? 32 : 2048) >> 4;
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;           // acc_phase: bit b = parity of accumulator b
      bool ok = true;
      const int steps = p.steps * p.segments;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        if (!mbar_wait(&acc_empty[buf], ((acc_phase >> buf) & 1u) ^ 1u, p.err)) break;
        fence_after();
        const uint32_t d = tmem + 256u * buf;
        for (int k = 0; k < steps; ++k) {
          if (!mbar_wait(&full[stage], phase, p.err)) { ok = false; break; }
          fence_after();
          if (lead) {
            const uint64_t at = static_cast<uint64_t>(stage * (kStage >> 4));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_bf16_pair(d, da + at + j * kStepA, db + at + j * kStepB, idesc<MODE>(), k > 0 || j > 0 ? 1u : 0u);
            commit2_both(&empty[stage]);
          }
          __syncwarp();
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (lead) commit2_both(&acc_full[buf]);
        __syncwarp();
        acc_phase ^= 1u << buf;
        buf ^= 1;
      }
      // the peer's last arrivals here have landed (see cluster_sync)
      for (int b = 0; b < 2; ++b) mbar_wait(&acc_empty[b], ((acc_phase >> b) & 1u) ^ 1u, p.err);
      if (lead) {
        commit2_lead(drain);
        mbar_wait(drain, 0, p.err);
      }
      __syncwarp();
    }
  } else {
    const int q = warp & 3;
    uint8_t* stg_warp = stg + q * kStgWarp;
    uint8_t* stg_row = stg_warp + lane * kStgStride;
    int buf = 0;
    uint32_t acc_phase = 0;
    for (int tile = pair; tile < total; tile += npairs) {
      const int mat = tile / per_mat;
      int r, c;
      tile_at(tile - mat * per_mat, p.row_tiles, p.col_tiles, r, c);
      bool ok = true;
      if (lane == 0) ok = mbar_wait(&acc_full[buf], (acc_phase >> buf) & 1u, p.err);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      fence_after();
      const uint32_t trow = tmem + (static_cast<uint32_t>(32 * q) << 16) + 256u * buf;
      const int64_t row0 = static_cast<int64_t>(r) * 256 + rank * 128 + 32 * q;   // first row of this warp
      const int64_t col0 = static_cast<int64_t>(c) * (MODE == kForward ? 128 : 256);
      uint16_t* out = MODE == kGradW && mat ? p.out[1] : p.out[0];
#pragma unroll 1
      for (int h = 0; h < (MODE == kForward ? 2 : 4); ++h) {      // 64 output columns at a time
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = 64 * h + 32 * e;
          float v[32];
          tmem_ld(trow + at, v);
          if (MODE == kForward) {
            float u[32];
            tmem_ld(trow + 128 + at, u);
            tmem_ld_wait(v, u);
            const int64_t rb = row0 / 32, cb = (col0 + at) / 32;
            if (p.saved != nullptr && rb < p.sv_rb && cb < p.sv_cb &&
                NV_IDX(saved_at(rb, cb, p.sv_cb) + 1024 <= p.sv_rb * p.sv_cb * 1024)) {
              float* g = p.saved + saved_at(rb, cb, p.sv_cb) + 4 * lane;
              float* w = g + p.sv_rb * p.sv_cb * 1024;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                *reinterpret_cast<float4*>(g + 128 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                *reinterpret_cast<float4*>(w + 128 * i) = make_float4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = act_value(v[i], p.act) * u[i];
          } else {
            tmem_ld_wait(v);
          }
          if (h == (MODE == kForward ? 1 : 3) && e == 1) {
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(peer_u32(smem_u32(&acc_empty[buf]), 0));   // accumulator free
          }
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4*>(stg_row + (32 * e + i) * 2) =
                make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]), bf16x2(v[i + 4], v[i + 5]),
                           bf16x2(v[i + 6], v[i + 7]));
        }
        __syncwarp();
        // 32 rows x 128 bytes: 8 lanes a row (cols % 8 == 0: a lane's 8 are in or out)
        const int64_t col = col0 + 64 * h + 8 * (lane & 7);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + (lane >> 3);
          if (row0 + rr < p.rows && col < p.cols && NV_IDX(in_matrix(row0 + rr, col, 8, p.rows, p.cols, p.ldo)))
            *reinterpret_cast<uint4*>(out + (row0 + rr) * p.ldo + col) =
                *reinterpret_cast<const uint4*>(stg_warp + rr * kStgStride + 16 * (lane & 7));
        }
        __syncwarp();
      }
      acc_phase ^= 1u << buf;
      buf ^= 1;
    }
  }
  fence_before();
  __syncthreads();
  cluster_sync();                              // neither CTA leaves while its peer may still signal it
  if (warp == 1) {
    fence_after();
    tmem_dealloc<2>(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// dG = dH U act'(G), dU = dH act(G) from the saved fp32 projections: a warp
// takes a 32 x 32 block, a lane one of its rows; dH and the results pass
// through shared memory so that global memory sees 64-byte row pieces.  Bound
// by memory, 10 bytes read and 4 written per element: 213 to 227 us for 8192 x 11008
// (5.6 to 5.9 TB/s) with a block per warp and small CTAs, so that the loads of one
// run under the arithmetic of others; 271 us with as many CTAs as fit, each
// walking over blocks.
// ---------------------------------------------------------------------------
// A 16-byte load that is read once (does not stay in L1).
__device__ __forceinline__ float4 ld_stream_f4(const float* p) {
  float4 v;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}

constexpr int kBwdWarps = 4;
constexpr int kBwdStride = 32 * 2 + 16;

__global__ void __launch_bounds__(32 * kBwdWarps, 5)
gated_slope_kernel(const float* __restrict__ saved, int64_t n_rb, int64_t n_cb, const uint16_t* __restrict__ dh,
                   int64_t ld_dh, int64_t M, int64_t F, int act, uint16_t* __restrict__ dg,
                   uint16_t* __restrict__ du) {
  __shared__ __align__(16) uint8_t tile[kBwdWarps][2][32 * kBwdStride];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* t0 = tile[warp][0];
  uint8_t* t1 = tile[warp][1];
  const int64_t blocks = n_rb * n_cb;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * kBwdWarps + warp; b < blocks;
       b += static_cast<int64_t>(gridDim.x) * kBwdWarps) {
    const int64_t rb = b / n_cb, cb = b - rb * n_cb;
    const int64_t col = cb * 32 + 8 * (lane & 3);
    // the whole block's loads first: 10 KB in flight per warp
    float4 g[8], u[8];
    const float* src = saved + saved_at(rb, cb, n_cb) + 4 * lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = ld_stream_f4(src + 128 * i);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = ld_stream_f4(src + blocks * 1024 + 128 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = 8 * i + (lane >> 2);
      const int64_t row = rb * 32 + rr;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < M && col < F && NV_IDX(in_matrix(row, col, 8, M, F, ld_dh))) v = ld_nc_v4(dh + row * ld_dh + col);
      *reinterpret_cast<uint4*>(t0 + rr * kBwdStride + 16 * (lane & 3)) = v;
    }
    __syncwarp();
    uint32_t* mine0 = reinterpret_cast<uint32_t*>(t0 + lane * kBwdStride);
    uint32_t* mine1 = reinterpret_cast<uint32_t*>(t1 + lane * kBwdStride);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gv[4] = {g[i].x, g[i].y, g[i].z, g[i].w}, uv[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      const uint2 d2 = *reinterpret_cast<const uint2*>(mine0 + 2 * i);
      const float dv[4] = {__uint_as_float(d2.x << 16), __uint_as_float(d2.x & 0xFFFF0000u),
                           __uint_as_float(d2.y << 16), __uint_as_float(d2.y & 0xFFFF0000u)};
      float da[4], ds[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        act_value_slope(gv[j], act, da[j], ds[j]);
        ds[j] = dv[j] * uv[j] * ds[j];
        da[j] = dv[j] * da[j];
      }
      *reinterpret_cast<uint2*>(mine0 + 2 * i) = make_uint2(bf16x2(ds[0], ds[1]), bf16x2(ds[2], ds[3]));
      *reinterpret_cast<uint2*>(mine1 + 2 * i) = make_uint2(bf16x2(da[0], da[1]), bf16x2(da[2], da[3]));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = 8 * i + (lane >> 2);
      const int64_t row = rb * 32 + rr;
      if (row < M && col < F && NV_IDX(in_matrix(row, col, 8, M, F, F))) {
        *reinterpret_cast<uint4*>(dg + row * F + col) = *reinterpret_cast<const uint4*>(t0 + rr * kBwdStride + 16 * (lane & 3));
        *reinterpret_cast<uint4*>(du + row * F + col) = *reinterpret_cast<const uint4*>(t1 + rr * kBwdStride + 16 * (lane & 3));
      }
    }
    __syncwarp();
  }
}

template <Mode MODE>
cudaError_t launch_pair(const CUtensorMap (&m)[4], Params& p, cudaStream_t s) {
  static bool attr_done[kMaxAttrDevices] = {};
  cudaError_t e = set_max_smem(gated_pair_kernel<MODE>, kSmem, attr_done);
  if (e != cudaSuccess) return e;
  p.row_tiles = static_cast<int>((p.rows + 255) / 256);
  p.col_tiles = static_cast<int>((p.cols + (MODE == kForward ? 127 : 255)) / (MODE == kForward ? 128 : 256));
  const int64_t tiles = static_cast<int64_t>(p.row_tiles) * p.col_tiles * p.mats;
  if (tiles == 0) return cudaSuccess;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const int64_t pairs = tiles < sm_count() / 2 ? tiles : sm_count() / 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  e = launch_k(gated_pair_kernel<MODE>, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads), kSmem, s, attr, 1, m[0],
               m[1], m[2], m[3], p);
  return e;
}

// Maps of a bf16 matrix [rows, cols]: K-major operand tiles (128 rows x 64),
// or MN-major ones (64 rows x 64).
bool map_k(CUtensorMap* m, const uint16_t* p, int64_t rows, int64_t cols, int64_t ld) {
  return map_bytes(m, p, rows, 2 * cols, 2 * ld, 128);
}
bool map_mn(CUtensorMap* m, const uint16_t* p, int64_t rows, int64_t cols, int64_t ld) {
  return map_bytes(m, p, rows, 2 * cols, 2 * ld, 64);
}

}  // namespace

size_t gated_saved_bytes(int64_t M, int64_t F) {
  return static_cast<size_t>((M + 31) / 32) * ((F + 31) / 32) * 1024 * 2 * sizeof(float);
}

cudaError_t launch_gated_forward(const GatedArgs& a, uint16_t* h, int64_t ldh, float* saved, cudaStream_t s) {
  CUtensorMap m[4];
  if (!map_k(&m[0], a.x, a.M, a.K, a.ldx) || !map_k(&m[2], a.w_gate, a.F, a.K, a.ldw) ||
      !map_k(&m[3], a.w_up, a.F, a.K, a.ldw))
    return cudaErrorInvalidValue;
  m[1] = m[0];
  Params p{};
  p.rows = a.M;
  p.cols = a.F;
  p.steps = static_cast<int>((a.K + 63) / 64);
  p.segments = 1;
  p.mats = 1;
  p.act = a.act;
  p.out[0] = h;
  p.ldo = ldh;
  p.saved = saved;
  p.sv_rb = (a.M + 31) / 32;
  p.sv_cb = (a.F + 31) / 32;
  p.err = a.err;
  return launch_pair<kForward>(m, p, s);
}

cudaError_t launch_gated_slope(const GatedArgs& a, const float* saved, const uint16_t* dh, int64_t ld_dh,
                               uint16_t* dg, uint16_t* du, cudaStream_t s) {
  const int64_t rb = (a.M + 31) / 32, cb = (a.F + 31) / 32;
  const int64_t ctas = (rb * cb + kBwdWarps - 1) / kBwdWarps, cap = 0x7FFFFFFF;
  const cudaError_t e = launch_k(gated_slope_kernel, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)),
                                 dim3(32 * kBwdWarps), 0, s, nullptr, 0, saved, rb, cb, dh, ld_dh, a.M, a.F, a.act, dg,
                                 du);
  return e;
}

cudaError_t launch_gated_grad_x(const GatedArgs& a, const uint16_t* dg, const uint16_t* du, uint16_t* dx,
                                int64_t ld_dx, cudaStream_t s) {
  CUtensorMap m[4];
  if (!map_k(&m[0], dg, a.M, a.F, a.F) || !map_k(&m[1], du, a.M, a.F, a.F) ||
      !map_mn(&m[2], a.w_gate, a.F, a.K, a.ldw) || !map_mn(&m[3], a.w_up, a.F, a.K, a.ldw))
    return cudaErrorInvalidValue;
  Params p{};
  p.rows = a.M;
  p.cols = a.K;
  p.steps = static_cast<int>((a.F + 63) / 64);
  p.segments = 2;
  p.mats = 1;
  p.out[0] = dx;
  p.ldo = ld_dx;
  p.err = a.err;
  return launch_pair<kGradX>(m, p, s);
}

cudaError_t launch_gated_grad_w(const GatedArgs& a, const uint16_t* dg, const uint16_t* du, uint16_t* dw_gate,
                                uint16_t* dw_up, cudaStream_t s) {
  // the matrices asked for, in the order gate, up
  const uint16_t* from[2] = {dw_gate != nullptr ? dg : du, du};
  CUtensorMap m[4];
  if (!map_mn(&m[0], from[0], a.M, a.F, a.F) || !map_mn(&m[1], from[1], a.M, a.F, a.F) ||
      !map_mn(&m[2], a.x, a.M, a.K, a.ldx))
    return cudaErrorInvalidValue;
  m[3] = m[2];
  Params p{};
  p.rows = a.F;
  p.cols = a.K;
  p.steps = static_cast<int>((a.M + 63) / 64);
  p.segments = 1;
  p.mats = (dw_gate != nullptr) + (dw_up != nullptr);
  p.out[0] = dw_gate != nullptr ? dw_gate : dw_up;
  p.out[1] = dw_up;
  p.ldo = a.K;
  p.err = a.err;
  return launch_pair<kGradW>(m, p, s);
}

NV_DEFINE_BOUNDS_READER(bounds_flags_gated)

}  // namespace nvfp4

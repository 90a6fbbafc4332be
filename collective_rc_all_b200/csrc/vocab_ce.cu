// vocab_ce.cu -- softmax cross entropy over a vocabulary cut into the ranks'
// pieces (the tensor-parallel output head), and its gradients, without
// keeping the logits.
//
// Page: "分布式训练/推理", the tensor-parallel sections (a linear layer's weight
// rows split over the ranks, the partial results joined by an all-reduce).
// With h [N, D], rank r's rows W_r of W [V, D], targets y:
//   z = h W^T,  lse_i = log sum_v exp z_iv,  loss_i = lse_i - z_{i, y_i}
//   G_iv = dloss_i (exp(z_iv - lse_i) - [v = y_i]),  dh = G W,  dW_r = G_r^T h
// The join over the ranks is a join over tiles: each 256-column tile of z
// leaves a (max, sum of exp) pair per row, and the pairs of all tiles of all
// ranks are merged in tile order; dh sums over the ranks' columns in order.
//
// Everything of size N V D is a bf16 tensor-core product with fp32
// accumulators; the logits live in tensor memory only.  The gradients'
// pass goes over the vocabulary in pieces of a few thousand columns: it
// computes the piece's logits again, writes G for the piece as bf16, and feeds
// it to the two products dW_r = G^T h (complete for the piece) and dh += G W
// (fp32 sums in the workspace, rounded once at the end).
//
// Rounding G to bf16 (2^-9 relative at most on average, independent from
// entry to entry) adds about as much error as the gradients' own rounding to
// bf16.  With few tokens one entry, the target's, carries a row's whole
// gradient and its rounding would show in every output of the row; there G is
// kept as the sum of two bf16 planes (2^-17).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "tc.cuh"

namespace rc {

// Number of bounded waits of this file's kernels that gave up.
__device__ unsigned int g_wait_timeouts_ce = 0;

namespace {

constexpr int kNT = 256;       // copy warp, product warp, two idle, four epilogue warps
constexpr int kBM = 128;       // rows of a tile (tensor-memory lanes)
constexpr int kBN = 256;       // columns of a tile
constexpr int kBK = 64;        // one 128-byte row of bf16
constexpr int kStages = 4;
constexpr uint32_t kABytes = kBM * kBK * 2;
constexpr uint32_t kBBytes = kBN * kBK * 2;
constexpr uint32_t kStageBytes = kABytes + kBBytes;
constexpr uint32_t kSmemBytes = kStages * kStageBytes + 1024;  // + slack to align to 1024
constexpr int kGroupM = 16;    // row tiles that share a sweep over the columns (L2 reuse)
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

enum Mode : int {
  kStats = 0,  // z tile -> (max, sum exp) per row, target logit
  kGrad = 1,   // z tile -> G tile
  kDW = 2,     // G^T h -> dW rows
  kDH = 3,     // G W -> fp32 sums
};

struct alignas(64) CeParams {
  CUtensorMap a;              // kStats, kGrad: h (K-major); kDW: G (64 x 64 boxes); kDH: G (K-major)
  CUtensorMap b[kMaxRanks];   // kStats, kGrad: W_r (K-major); kDW: h (64 x 64 boxes, b[0]); kDH: W_r (64 x 64 boxes)
  int rows[kMaxRanks];        // rows of each rank's piece
  char *dw[kMaxRanks];        // kDW
  const int32_t *target;
  const float *lse_in, *dloss;  // kGrad
  float2 *part;               // kStats: [tile][N]
  float *ztarget;             // kStats: [N]
  char *g;                    // kGrad: [planes][N][gcols] bf16
  float *dh;                  // kDH: [splits][N][dpad]
  int64_t N, V;
  int D, dpad;
  int C;                      // rows of a full rank piece
  int tpr;                    // 256-row tiles per rank
  int j0;                     // first tile of this launch's piece
  int gcols;                  // columns of G (the piece's, a multiple of 256)
  int planes;                 // bf16 planes of G
  int mt, nt, nk, kper, splits;
  int64_t tiles;
  int ignore;
  bool first;                 // kDH: store instead of add
  bool dw_vec;                // kDW: rows can be written as 16-byte vectors
};

struct TileAt {
  int m, n, s;
};

// Tiles go in groups of kGroupM row tiles, all columns of a group before the
// next group; the splits of k are outermost.
__device__ __forceinline__ TileAt tile_at(const CeParams &a, int64_t t) {
  const int64_t per = (int64_t)a.mt * a.nt;
  TileAt r;
  r.s = (int)(t / per);
  const int64_t u = t - r.s * per;
  const int64_t gsz = (int64_t)kGroupM * a.nt;
  const int g = (int)(u / gsz);
  const int64_t w = u - g * gsz;
  const int gm = min(kGroupM, a.mt - g * kGroupM);
  r.n = (int)(w / gm);
  r.m = g * kGroupM + (int)(w - (int64_t)r.n * gm);
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Flow {
  volatile uint32_t *dead;
  __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
      if (*dead) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        if (atomicExch(const_cast<uint32_t *>(dead), 1u) == 0) atomicAdd(&g_wait_timeouts_ce, 1u);
        return false;
      }
    }
    return true;
  }
};

template <int MODE>
__global__ void __launch_bounds__(kNT, 1) rc_ce_gemm_kernel(const __grid_constant__ CeParams a) {
  constexpr bool A_MN = MODE == kDW;
  constexpr bool B_MN = MODE == kDW || MODE == kDH;
  extern __shared__ char smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_base_s;
  __shared__ uint32_t dead_s;
  const uint32_t smem0 = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 128);
    }
    mbar_init(&drained, 1);
    dead_s = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc_all(&tmem_base_s);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_base_s;
  const Flow flow{&dead_s};
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < a.tiles; t += gridDim.x) {
        const TileAt w = tile_at(a, t);
        const int k0 = w.s * a.kper, k1 = min(a.nk, k0 + a.kper);
        for (int k = k0; k < k1; ++k, ++it) {
          const uint32_t slot = it % kStages;
          if (it >= kStages && !flow.wait(&empty[slot], (it / kStages - 1) & 1)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem0 + slot * kStageBytes, sb = sa + kABytes;
          mbar_arrive_expect_tx(&full[slot], kStageBytes);
          if constexpr (MODE == kStats || MODE == kGrad) {
            const int j = a.j0 + w.n, r = j / a.tpr;
            tma_load_2d(sa, &a.a, k * kBK, w.m * kBM, &full[slot]);
            tma_load_2d(sb, &a.b[r], k * kBK, (j - r * a.tpr) * kBN, &full[slot]);
          } else if constexpr (MODE == kDW) {
            const int per = a.nk / a.planes, plane = k / per, kk = k - plane * per;
#pragma unroll
            for (int i = 0; i < kBM / 64; ++i)
              tma_load_3d(sa + i * 8192, &a.a, w.m * kBM + i * 64, kk * kBK, plane, &full[slot]);
#pragma unroll
            for (int i = 0; i < kBN / 64; ++i)
              tma_load_2d(sb + i * 8192, &a.b[0], w.n * kBN + i * 64, kk * kBK, &full[slot]);
          } else {
            const int per = a.nk / a.planes, plane = k / per, kk = k - plane * per;
            const int j = a.j0 + kk * kBK / kBN, r = j / a.tpr;
            const int row = (j - r * a.tpr) * kBN + kk * kBK % kBN;
            tma_load_3d(sa, &a.a, kk * kBK, w.m * kBM, plane, &full[slot]);
#pragma unroll
            for (int i = 0; i < kBN / 64; ++i)
              tma_load_2d(sb + i * 8192, &a.b[r], w.n * kBN + i * 64, row, &full[slot]);
          }
        }
      }
      if (!ok) {  // wait (bounded) for this block's copies in flight
        const uint32_t n = it < kStages ? it : kStages;
        for (uint32_t i = it - n; i < it; ++i)
          mbar_wait_bounded(&full[i % kStages], (i / kStages) & 1, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = tc_idesc(kBM, kBN, A_MN, B_MN);
      constexpr uint32_t a_step = (A_MN ? 2048 : 32) >> 4, b_step = (B_MN ? 2048 : 32) >> 4;
      uint32_t it = 0, i = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < a.tiles; t += gridDim.x, ++i) {
        const TileAt w = tile_at(a, t);
        const int k0 = w.s * a.kper, k1 = min(a.nk, k0 + a.kper);
        const uint32_t acc = i & 1, d = tmem + acc * kBN;
        if (i >= 2 && !flow.wait(&acc_empty[acc], (i / 2 - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        for (int k = k0; k < k1; ++k, ++it) {
          const uint32_t slot = it % kStages;
          if (!flow.wait(&full[slot], (it / kStages) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sa = smem0 + slot * kStageBytes, sb = sa + kABytes;
          const uint64_t da = tc_desc(sa, A_MN ? 8192 : 16), db = tc_desc(sb, B_MN ? 8192 : 16);
#pragma unroll
          for (int q = 0; q < kBK / 16; ++q)
            tc_mma(d, da + q * a_step, db + q * b_step, idesc, k > k0 || q > 0);
          tc_commit(&empty[slot]);
        }
        if (ok) tc_commit(&acc_full[acc]);
      }
      if (!ok) {  // the products in flight read shared memory and write tensor memory
        tc_commit(&drained);
        mbar_wait_bounded(&drained, 0, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int quad = warp & 3;
    uint32_t i = 0;
    for (int64_t t = blockIdx.x; t < a.tiles; t += gridDim.x, ++i) {
      const TileAt w = tile_at(a, t);
      const uint32_t acc = i & 1;
      const int64_t row = (int64_t)w.m * kBM + quad * 32 + lane;  // row of this thread (kDW: column of G)
      if (!__all_sync(0xffffffffu, flow.wait(&acc_full[acc], (i / 2) & 1))) break;
      tc_fence_after_sync();
      const uint32_t src = tmem + acc * kBN + ((uint32_t)(quad * 32) << 16);
      if constexpr (MODE == kStats || MODE == kGrad) {
        const int j = a.j0 + w.n, r = j / a.tpr, v0 = (j - r * a.tpr) * kBN;
        const int cols = max(0, min(kBN, a.rows[r] - v0));
        const bool live = row < a.N;
        const int y = live ? a.target[row] : 0;
        const int64_t yt = (int64_t)y - ((int64_t)r * a.C + v0);  // the target's column in this tile, if it is in it
        const int ycol = (y != a.ignore && yt >= 0 && yt < cols) ? (int)yt : -1;
        if constexpr (MODE == kStats) {
          float m = -INFINITY, s = 0.0f, zt = 0.0f;
#pragma unroll 1
          for (int c = 0; c < kBN; c += 32) {
            float z[32];
            tmem_load32(src + c, z);
            if (c + 32 > cols) {
#pragma unroll
              for (int q = 0; q < 32; ++q) z[q] = c + q < cols ? z[q] : -INFINITY;
            }
            if ((ycol & ~31) == c) {
#pragma unroll
              for (int q = 0; q < 32; ++q) zt = (ycol & 31) == q ? z[q] : zt;
            }
            float cm = z[0];
#pragma unroll
            for (int q = 1; q < 32; ++q) cm = fmaxf(cm, z[q]);
            const float nm = fmaxf(m, cm);
            const float base = nm > -INFINITY ? nm * kLog2e : 0.0f;
            float cs = 0.0f;
#pragma unroll
            for (int q = 0; q < 32; ++q) cs += ex2(fmaf(z[q], kLog2e, -base));
            s = fmaf(s, ex2(fmaf(m, kLog2e, -base)), cs);
            m = nm;
          }
          if (live) {
            a.part[(int64_t)j * a.N + row] = make_float2(m, s);
            if (ycol >= 0) a.ztarget[row] = zt;
          }
        } else {
          const float lse2 = live ? a.lse_in[row] * kLog2e : 0.0f;
          float g = live ? a.dloss[row] : 0.0f;
          // a label that is no word and not the ignored one poisons its row
          if (y < 0 || y >= a.V) g = __int_as_float(0x7fc00000);
          const bool zero = !live || y == a.ignore;
          char *out = a.g + ((int64_t)row * a.gcols + (int64_t)w.n * kBN) * 2;
          const int64_t plane = a.N * (int64_t)a.gcols * 2;
#pragma unroll 1
          for (int c = 0; c < kBN; c += 32) {
            float z[32];
            tmem_load32(src + c, z);
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              float pr = ex2(fmaf(z[q], kLog2e, -lse2));
              pr -= c + q == ycol ? 1.0f : 0.0f;
              z[q] = (zero || c + q >= cols) ? 0.0f : pr * g;
            }
            if (live) {
#pragma unroll
              for (int q = 0; q < 32; q += 8) {
                uint32_t hi[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) hi[u] = pack_bf16x2(z[q + 2 * u], z[q + 2 * u + 1]);
                st_v4(out + (c + q) * 2, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                if (a.planes == 2) {
                  uint32_t lo[4];
#pragma unroll
                  for (int u = 0; u < 4; ++u)
                    lo[u] = pack_bf16x2(z[q + 2 * u] - __uint_as_float(hi[u] << 16),
                                        z[q + 2 * u + 1] - __uint_as_float(hi[u] & 0xffff0000u));
                  st_v4(out + plane + (c + q) * 2, make_uint4(lo[0], lo[1], lo[2], lo[3]));
                }
              }
            }
          }
        }
      } else if constexpr (MODE == kDW) {
        const int j = a.j0 + w.m / 2, r = j / a.tpr;
        const int v = (j - r * a.tpr) * kBN + (w.m & 1) * kBM + quad * 32 + lane;
        const bool live = v < a.rows[r];
        char *out = a.dw[r] + ((int64_t)v * a.D + (int64_t)w.n * kBN) * 2;
        const int cols = min(kBN, a.D - w.n * kBN);
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          float z[32];
          tmem_load32(src + c, z);
          if (!live) continue;
          if (a.dw_vec) {
#pragma unroll
            for (int q = 0; q < 32; q += 8)
              if (c + q < cols)
                st_v4(out + (c + q) * 2, make_uint4(pack_bf16x2(z[q], z[q + 1]), pack_bf16x2(z[q + 2], z[q + 3]),
                                                    pack_bf16x2(z[q + 4], z[q + 5]), pack_bf16x2(z[q + 6], z[q + 7])));
          } else {
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (c + q < cols) store_elem<BF16>(out, c + q, z[q]);
          }
        }
      } else {
        const bool live = row < a.N;
        float *out = a.dh + ((int64_t)w.s * a.N + row) * a.dpad + (int64_t)w.n * kBN;
        const int cols = min(kBN, a.dpad - w.n * kBN);  // a multiple of 8
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          float z[32];
          tmem_load32(src + c, z);
          if (!live) continue;
#pragma unroll
          for (int q = 0; q < 32; q += 4) {
            if (c + q < cols) {
              float4 *o = reinterpret_cast<float4 *>(out + c + q);
              float4 v = make_float4(z[q], z[q + 1], z[q + 2], z[q + 3]);
              if (!a.first) {
                const float4 u = *o;
                v = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
              }
              *o = v;
            }
          }
        }
      }
      tc_fence_before_sync();
      mbar_arrive(&acc_empty[acc]);
    }
  }
  __syncthreads();
  if (warp == 2) tmem_free_all(tmem);
}

// Joins the tiles' (max, sum) pairs of each row in a fixed order:
// a block has 2^lg rows and 256 / 2^lg threads per row.
__global__ void __launch_bounds__(kNT) rc_ce_join_kernel(const float2 *part, const float *ztarget,
                                                         const int32_t *target, float *loss, float *lse, int64_t N,
                                                         int64_t V, int tiles, int lg, int ignore) {
  __shared__ float sm[kNT], ss[kNT];
  pdl_wait();
  const int rx = threadIdx.x & ((1 << lg) - 1), ty = threadIdx.x >> lg, nty = kNT >> lg;
  const int64_t row = ((int64_t)blockIdx.x << lg) + rx;
  float m = -INFINITY, s = 0.0f;
  if (row < N) {
    for (int t = ty; t < tiles; t += nty) {
      const float2 v = part[(int64_t)t * N + row];
      const float nm = fmaxf(m, v.x);
      const float base = nm > -INFINITY ? nm : 0.0f;
      s = s * expf(m - base) + v.y * expf(v.x - base);
      m = nm;
    }
  }
  sm[threadIdx.x] = m;
  ss[threadIdx.x] = s;
  __syncthreads();
  for (int h = nty / 2; h > 0; h >>= 1) {
    if (ty < h) {
      const int o = threadIdx.x + (h << lg);
      const float nm = fmaxf(sm[threadIdx.x], sm[o]);
      const float base = nm > -INFINITY ? nm : 0.0f;
      ss[threadIdx.x] = ss[threadIdx.x] * expf(sm[threadIdx.x] - base) + ss[o] * expf(sm[o] - base);
      sm[threadIdx.x] = nm;
    }
    __syncthreads();
  }
  if (ty == 0 && row < N) {
    const float l = sm[rx] + logf(ss[rx]);
    const int y = target[row];
    lse[row] = l;
    // a label outside [0, V) that is not the ignored one has no loss
    loss[row] = y == ignore ? 0.0f : (y < 0 || y >= V) ? __int_as_float(0x7fc00000) : l - ztarget[row];
  }
}

// dst[row][0, dpad) = src[row][0, D), zero behind D, and zero in rows whose
// target is ignored (target NULL: none), so that whatever a padded row holds
// stays out of the products.
__global__ void __launch_bounds__(kNT) rc_ce_pack_kernel(const uint16_t *src, uint16_t *dst, const int32_t *target,
                                                         int64_t rows, int D, int dpad, int ignore) {
  pdl_wait();
  const int per = dpad / 8;
  const int64_t n = rows * per;
  for (int64_t u = (int64_t)blockIdx.x * kNT + threadIdx.x; u < n; u += (int64_t)gridDim.x * kNT) {
    const int64_t row = u / per;
    const int c = (int)(u - row * per) * 8;
    const bool skip = target != nullptr && target[row] == ignore;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int x = c + 2 * q;
      const uint32_t lo = !skip && x < D ? src[row * D + x] : 0u;
      const uint32_t hi = !skip && x + 1 < D ? src[row * D + x + 1] : 0u;
      w[q] = lo | (hi << 16);
    }
    st_v4(dst + row * dpad + c, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// dh = bf16(sum of the splits' sums, in order).
__global__ void __launch_bounds__(kNT) rc_ce_finish_kernel(const float *sums, char *dh, int64_t N, int D, int dpad,
                                                           int splits) {
  pdl_wait();
  const int64_t n = N * D;
  for (int64_t u = (int64_t)blockIdx.x * kNT + threadIdx.x; u < n; u += (int64_t)gridDim.x * kNT) {
    const int64_t row = u / D;
    const float *at = sums + row * dpad + (u - row * D);
    float v = at[0];
    for (int s = 1; s < splits; ++s) v += at[(int64_t)s * N * dpad];
    store_elem<BF16>(dh, u, v);
  }
}

// ---------------------------------------------------------------- host side
typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static EncodeFn fn = []() -> EncodeFn {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A bf16 matrix [planes][rows][cols], `pitch` elements from row to row, read
// in boxes of 64 columns x box_rows rows with the 128-byte swizzle; what lies
// outside reads as zero.
bool make_map(CUtensorMap *map, const void *base, int64_t planes, int64_t rows, int64_t cols, int64_t pitch,
              int box_rows) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const int rank = planes > 0 ? 3 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)std::max<int64_t>(planes, 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)pitch * 2 * (cuuint64_t)rows};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }

// How a problem is cut, and where its parts lie in the workspace.
struct Plan {
  int C, tpr, ranks, tiles;       // rank pieces, 256-row tiles per rank, ranks with rows, all tiles
  int dpad;
  int planes, per_piece, pieces;  // of the gradients' pass
  int splits, kper;
  size_t off_part, off_zt, off_h, off_w, off_g, off_dh, bytes;
};

Plan make_plan(const CeShape &s, bool backward, bool copies) {
  Plan q{};
  q.C = (int)cdiv(s.vocab, s.p);
  q.tpr = (int)cdiv(q.C, kBN);
  q.ranks = (int)cdiv(s.vocab, q.C);
  q.tiles = q.ranks * q.tpr;
  q.dpad = (int)up(s.d, 8);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 1023) & ~(size_t)1023;
    return here;
  };
  const size_t N = (size_t)s.tokens;
  if (copies || backward) q.off_h = take(N * q.dpad * 2);
  if (copies) q.off_w = take((size_t)q.ranks * q.C * q.dpad * 2);
  if (!backward) {
    q.off_part = take((size_t)q.tiles * N * 8);
    q.off_zt = take(N * 4);
  } else {
    // two planes up to 128 tokens: one row tile, whose products take less
    // time than reading the weights even when there are twice as many
    q.planes = s.tokens <= kBM ? 2 : 1;
    const int64_t tile_bytes = (int64_t)q.planes * s.tokens * kBN * 2;
    const int64_t want = std::max<int64_t>(16, (64ll << 20) / tile_bytes);
    q.pieces = (int)cdiv(q.tiles, std::min<int64_t>(want, q.tiles));
    q.per_piece = (int)cdiv(q.tiles, q.pieces);
    q.pieces = (int)cdiv(q.tiles, q.per_piece);
    // few output tiles of dh: split its long k (the piece's columns)
    const int64_t nk = (int64_t)q.planes * q.per_piece * (kBN / kBK);
    const int64_t out_tiles = cdiv(s.tokens, kBM) * cdiv(s.d, kBN);
    int64_t sp = std::max<int64_t>(1, std::min<int64_t>(device_sm_count() / out_tiles, nk / 8));
    q.kper = (int)cdiv(nk, sp);
    q.splits = (int)cdiv(nk, q.kper);
    q.off_g = take((size_t)q.planes * N * q.per_piece * kBN * 2);
    q.off_dh = take((size_t)q.splits * N * q.dpad * 4);
  }
  q.bytes = at;
  return q;
}

template <int MODE>
cudaError_t gemm(CeParams &a, cudaStream_t s) {
  cudaError_t err = cudaFuncSetAttribute(rc_ce_gemm_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
  if (err != cudaSuccess) return err;
  if (a.splits < 1) {
    a.splits = 1;
    a.kper = a.nk;
  }
  a.tiles = (int64_t)a.mt * a.nt * a.splits;
  const int64_t grid = std::min<int64_t>(a.tiles, device_sm_count());
  return launch_kernel(rc_ce_gemm_kernel<MODE>, dim3((unsigned)grid), dim3(kNT), kSmemBytes, s, a);
}

cudaError_t pack(const void *src, void *dst, const int32_t *target, int64_t rows, int D, int dpad, int ignore,
                 cudaStream_t s) {
  const int64_t n = rows * (dpad / 8);
  const int64_t grid = std::min<int64_t>(cdiv(n, kNT), (int64_t)device_sm_count() * 8);
  return launch_kernel(rc_ce_pack_kernel, dim3((unsigned)grid), dim3(kNT), 0, s,
                       static_cast<const uint16_t *>(src), static_cast<uint16_t *>(dst), target, rows, D, dpad,
                       ignore);
}

// Whether the tiled copies can read the caller's buffers (16-byte bases and
// rows); otherwise they read copies in the workspace.
bool copies_needed(const CeJob &j) {
  bool ok = j.shape.d % 8 == 0 && reinterpret_cast<uintptr_t>(j.hidden) % 16 == 0;
  for (int r = 0; r < j.shape.p; ++r) ok = ok && reinterpret_cast<uintptr_t>(j.weight[r]) % 16 == 0;
  return !ok;
}

struct Operands {
  const char *h;
  const char *w[kMaxRanks];
  int pitch;
};

// The operands as the products read them, copied where that is needed.
cudaError_t operands(const CeJob &j, const Plan &q, bool copies, Operands *o, int *rows, cudaStream_t s) {
  char *ws = static_cast<char *>(j.ws);
  cudaError_t err;
  o->pitch = copies ? q.dpad : j.shape.d;
  o->h = static_cast<const char *>(j.hidden);
  if (copies || j.backward) {
    if ((err = pack(j.hidden, ws + q.off_h, j.backward ? j.target : nullptr, j.shape.tokens, j.shape.d, q.dpad,
                    j.ignore, s)) != cudaSuccess)
      return err;
    o->h = ws + q.off_h;
  }
  for (int r = 0; r < q.ranks; ++r) {
    rows[r] = (int)std::min<int64_t>(q.C, j.shape.vocab - (int64_t)r * q.C);
    o->w[r] = static_cast<const char *>(j.weight[r]);
    if (copies) {
      char *dst = ws + q.off_w + (size_t)r * q.C * q.dpad * 2;
      if ((err = pack(j.weight[r], dst, nullptr, rows[r], j.shape.d, q.dpad, 0, s)) != cudaSuccess) return err;
      o->w[r] = dst;
    }
  }
  return cudaSuccess;
}

}  // namespace

size_t ce_workspace(const CeShape &s, bool backward, bool copies) { return make_plan(s, backward, copies).bytes; }
size_t ce_workspace(const CeJob &j) { return make_plan(j.shape, j.backward, copies_needed(j)).bytes; }

cudaError_t launch_ce_forward(const CeJob &j, cudaStream_t s) {
  const bool copies = copies_needed(j);
  const Plan q = make_plan(j.shape, false, copies);
  char *ws = static_cast<char *>(j.ws);
  CeParams a{};
  Operands o{};
  cudaError_t err;
  if ((err = operands(j, q, copies, &o, a.rows, s)) != cudaSuccess) return err;
  const int D = j.shape.d;
  const int64_t N = j.shape.tokens;
  if (!make_map(&a.a, o.h, 0, N, D, o.pitch, kBM)) return cudaErrorInvalidValue;
  for (int r = 0; r < q.ranks; ++r)
    if (!make_map(&a.b[r], o.w[r], 0, a.rows[r], D, o.pitch, kBN)) return cudaErrorInvalidValue;
  a.target = j.target;
  a.part = reinterpret_cast<float2 *>(ws + q.off_part);
  a.ztarget = reinterpret_cast<float *>(ws + q.off_zt);
  a.N = N;
  a.D = D;
  a.C = q.C;
  a.tpr = q.tpr;
  a.ignore = j.ignore;
  a.mt = (int)cdiv(N, kBM);
  a.nt = q.tiles;
  a.nk = (int)cdiv(D, kBK);
  if ((err = gemm<kStats>(a, s)) != cudaSuccess) return err;
  // as many rows per block as leave every thread of a row a tile or more
  int lg = 5;
  while (lg > 0 && ((kNT >> lg) < q.tiles && (1 << (lg - 1)) >= N)) --lg;
  return launch_kernel(rc_ce_join_kernel, dim3((unsigned)cdiv(N, 1 << lg)), dim3(kNT), 0, s,
                       (const float2 *)a.part, (const float *)a.ztarget, j.target, j.loss, j.lse, N,
                       (int64_t)j.shape.vocab, q.tiles, lg, j.ignore);
}

cudaError_t launch_ce_backward(const CeJob &j, cudaStream_t s) {
  const bool copies = copies_needed(j);
  const Plan q = make_plan(j.shape, true, copies);
  char *ws = static_cast<char *>(j.ws);
  CeParams base{};
  Operands o{};
  cudaError_t err;
  if ((err = operands(j, q, copies, &o, base.rows, s)) != cudaSuccess) return err;
  const int D = j.shape.d;
  const int64_t N = j.shape.tokens;
  base.target = j.target;
  base.lse_in = j.lse_in;
  base.dloss = j.dloss;
  base.g = ws + q.off_g;
  base.dh = reinterpret_cast<float *>(ws + q.off_dh);
  base.N = N;
  base.D = D;
  base.dpad = q.dpad;
  base.C = q.C;
  base.tpr = q.tpr;
  base.planes = q.planes;
  base.ignore = j.ignore;
  base.V = j.shape.vocab;
  base.dw_vec = D % 8 == 0;
  for (int r = 0; r < q.ranks; ++r) {
    base.dw[r] = static_cast<char *>(j.dweight[r]);
    base.dw_vec = base.dw_vec && reinterpret_cast<uintptr_t>(j.dweight[r]) % 16 == 0;
  }
  CeParams z = base, w = base, h = base;
  if (!make_map(&z.a, o.h, 0, N, D, q.dpad, kBM) || !make_map(&w.b[0], o.h, 0, N, D, q.dpad, 64))
    return cudaErrorInvalidValue;
  for (int r = 0; r < q.ranks; ++r)
    if (!make_map(&z.b[r], o.w[r], 0, base.rows[r], D, o.pitch, kBN) ||
        !make_map(&h.b[r], o.w[r], 0, base.rows[r], D, o.pitch, 64))
      return cudaErrorInvalidValue;
  for (int i = 0; i < q.pieces; ++i) {
    const int j0 = i * q.per_piece, nt = std::min(q.per_piece, q.tiles - j0), cols = nt * kBN;
    z.j0 = w.j0 = h.j0 = j0;
    z.gcols = w.gcols = h.gcols = cols;
    if (!make_map(&w.a, base.g, q.planes, N, cols, cols, 64) || !make_map(&h.a, base.g, q.planes, N, cols, cols, kBM))
      return cudaErrorInvalidValue;
    z.mt = (int)cdiv(N, kBM);
    z.nt = nt;
    z.nk = (int)cdiv(D, kBK);
    if ((err = gemm<kGrad>(z, s)) != cudaSuccess) return err;
    w.mt = cols / kBM;
    w.nt = (int)cdiv(D, kBN);
    w.nk = q.planes * (int)cdiv(N, kBK);
    if ((err = gemm<kDW>(w, s)) != cudaSuccess) return err;
    h.mt = (int)cdiv(N, kBM);
    h.nt = (int)cdiv(D, kBN);
    h.nk = q.planes * cols / kBK;
    h.kper = q.kper;
    h.splits = (int)cdiv(h.nk, q.kper);
    h.first = i == 0;
    if ((err = gemm<kDH>(h, s)) != cudaSuccess) return err;
  }
  const int64_t grid = std::min<int64_t>(cdiv(N * D, kNT), (int64_t)device_sm_count() * 8);
  return launch_kernel(rc_ce_finish_kernel, dim3((unsigned)grid), dim3(kNT), 0, s, (const float *)base.dh,
                       static_cast<char *>(j.dhidden), N, D, q.dpad, q.splits);
}

cudaError_t read_and_clear_ce_timeouts(unsigned int *count) {
  unsigned int z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts_ce, sizeof z);
  if (e == cudaSuccess && *count) e = cudaMemcpyToSymbol(g_wait_timeouts_ce, &z, sizeof z);
  return e;
}

}  // namespace rc

// gate.cu -- the mixture-of-experts gate over p rank buffers: softmax over a
// token's router logits, the top-k experts, per-rank per-expert counts (the
// split counts of the dispatch), the balance loss over all ranks, and the
// gradient to the logits.
//
// Page: "分布式训练/推理", section "从路由结果到专家输出" (the router picks k
// experts per token; split counts tell the receivers how much arrives).  The
// balance loss is the usual one of sparse expert layers:
//   f_e = (tokens' choices of e) / (k M),  P_e = (1/M) sum_t p_te,
//   loss = coef * E * sum_e f_e P_e,  M = tokens that are not masked,
// over the tokens of all p ranks.  f_e is a count and carries no gradient:
//   dL/dp_te = dloss * coef * E * f_e / M (+ the chosen weights' gradients),
//   dz = p (dp - sum_e p dp).
//
// A token's row lies in the registers of LPT lanes, VPL values each (a lane
// owns VPL neighbouring experts), so a warp works on 32 / LPT tokens at once
// and every reduction over a row is log2(LPT) shuffles.  The sums over tokens
// (P_e, counts) stay in registers while a block walks its tokens and leave it
// as one partial per block; a second launch adds the partials in block order,
// so the results are the same on every run (no floating-point atomics).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace rc {
namespace {

constexpr int kNT = 256;
constexpr int kWarps = kNT / 32;

struct GateParams {
  const char *z[kMaxRanks];
  const uint8_t *mask[kMaxRanks];  // NULL: no token is masked
  int32_t *ids[kMaxRanks];
  float *w[kMaxRanks];
  int32_t *counts[kMaxRanks];
  const float *dw[kMaxRanks];  // backward; NULL: zero
  char *dz[kMaxRanks];
  float *part_p;      // [p * blocks][E]
  int32_t *part_c;    // [p * blocks][E]
  int32_t *part_m;    // [p * blocks]
  float *stats;       // f[E], P[E], M
  float *loss;
  const float *dloss;  // NULL: zero
  uint64_t tokens;
  int E, k, p, blocks;  // blocks: blocks per rank
  float coef;
  bool norm, vec;  // vec: rows are read and written as 16-byte vectors
};

// The row's values of this lane: experts [lane * VPL, lane * VPL + VPL);
// those past E read as -inf.
template <class T, int VPL>
__device__ __forceinline__ void load_row(const char *row, int e0, int E, bool vec, float (&z)[VPL]) {
  constexpr int V = kVec<T>;
  if (vec) {
#pragma unroll
    for (int j = 0; j < VPL; j += V) {
      if (e0 + j < E) {  // E is a multiple of V here
        float t[V];
        unpack<T>(ld_stream_v4(row + (uint64_t)(e0 + j) * T::kBytes), t);
#pragma unroll
        for (int i = 0; i < V; ++i) z[j + i] = t[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) z[j + i] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) z[j] = e0 + j < E ? load_elem<T>(row, e0 + j) : -INFINITY;
  }
}

template <int LPT>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = LPT / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The numbers' order as unsigned integers; 0 for -inf and NaN, which are never
// chosen.  -0 counts as +0, so that the two tie.
__device__ __forceinline__ uint32_t order_key(float z) {
  if (!(z > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(z + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// exp(z - max) of this lane's values, and the row's sum of them; a row of -inf
// alone (max = -inf) is all zeros.  A NaN, or +inf, makes the sum NaN.
template <int LPT, int VPL>
__device__ __forceinline__ float row_exp(const float (&z)[VPL], float (&ex)[VPL], bool *live) {
  float m = -INFINITY;
  int nan = 0;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    m = fmaxf(m, z[j]);
    nan |= isnan(z[j]) ? 1 : 0;
  }
  // every lane takes part in every shuffle, whatever it holds
#pragma unroll
  for (int d = LPT / 2; d > 0; d >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    nan |= __shfl_xor_sync(0xffffffffu, nan, d);
  }
  *live = m > -INFINITY || nan != 0;
  const float base = m > -INFINITY ? m : 0.0f;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    ex[j] = expf(z[j] - base);
    s += ex[j];
  }
  return row_sum<LPT>(s);
}

template <class T, int LPT, int VPL>
__global__ void __launch_bounds__(kNT) rc_gate_kernel(const __grid_constant__ GateParams a) {
  constexpr int TPW = 32 / LPT;  // tokens per warp and step
  __shared__ float sp[kWarps][LPT * VPL];
  __shared__ int32_t sc[kWarps][LPT * VPL];
  __shared__ int32_t sm[kWarps];
  pdl_wait();
  const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (LPT - 1), e0 = sub * VPL;
  float acc[VPL];
  int32_t cnt[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    acc[j] = 0.0f;
    cnt[j] = 0;
  }
  int32_t tokens = 0;
  const uint64_t step = (uint64_t)gridDim.x * kWarps * TPW;
  for (uint64_t t0 = ((uint64_t)blockIdx.x * kWarps + warp) * TPW; t0 < a.tokens; t0 += step) {
    const uint64_t t = t0 + lane / LPT;
    const bool have = t < a.tokens;
    const bool unmasked = have && (a.mask[r] == nullptr || a.mask[r][t] != 0);
    float z[VPL], ex[VPL];
    if (unmasked) {
      load_row<T, VPL>(a.z[r] + t * (uint64_t)a.E * T::kBytes, e0, a.E, a.vec, z);
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) z[j] = -INFINITY;
    }
    bool live;
    const float total = row_exp<LPT, VPL>(z, ex, &live);
    const float inv = live ? 1.0f / total : 0.0f;
    uint32_t key[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      key[j] = order_key(z[j]);
      ex[j] *= inv;  // the probability
      acc[j] += ex[j];
    }
    tokens += (live && sub == 0) ? 1 : 0;
    // k rounds: the lane's best (lowest index first), then the row's best
    float share = 0.0f;
    for (int i = 0; i < a.k; ++i) {
      uint32_t bk = 0;
      int bj = 0;
      float bp = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        if (key[j] > bk) {
          bk = key[j];
          bj = j;
          bp = ex[j];
        }
      }
      int be = e0 + bj;
#pragma unroll
      for (int d = LPT / 2; d > 0; d >>= 1) {
        const uint32_t ok = __shfl_xor_sync(0xffffffffu, bk, d);
        const int oe = __shfl_xor_sync(0xffffffffu, be, d);
        const float op = __shfl_xor_sync(0xffffffffu, bp, d);
        if (ok > bk || (ok == bk && oe < be)) {
          bk = ok;
          be = oe;
          bp = op;
        }
      }
      const bool found = bk != 0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        if (found && be == e0 + j) {
          key[j] = 0;
          cnt[j] += 1;
        }
      }
      share += found ? bp : 0.0f;
      // lane i % LPT writes slot i
      if (have && (i & (LPT - 1)) == sub) {
        a.ids[r][t * a.k + i] = found ? be : -1;
        a.w[r][t * a.k + i] = found ? bp : 0.0f;
      }
    }
    if (a.norm && have) {
      // the same lane that wrote the slot scales it
      for (int i = sub; i < a.k; i += LPT) {
        const float v = a.w[r][t * a.k + i];
        a.w[r][t * a.k + i] = share > 0.0f || isnan(share) ? v / share : 0.0f;
      }
    }
  }
  // lanes that own the same experts, then the block's warps
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
#pragma unroll
    for (int d = 16; d >= LPT; d >>= 1) {
      acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], d);
      cnt[j] += __shfl_xor_sync(0xffffffffu, cnt[j], d);
    }
    if (lane < LPT) {
      sp[warp][e0 + j] = acc[j];
      sc[warp][e0 + j] = cnt[j];
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) tokens += __shfl_xor_sync(0xffffffffu, tokens, d);
  if (lane == 0) sm[warp] = tokens;
  __syncthreads();
  const uint64_t b = (uint64_t)r * gridDim.x + blockIdx.x;
  for (int e = threadIdx.x; e < a.E; e += kNT) {
    float s = 0.0f;
    int32_t c = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      s += sp[w][e];
      c += sc[w][e];
    }
    a.part_p[b * a.E + e] = s;
    a.part_c[b * a.E + e] = c;
  }
  if (threadIdx.x == 0) {
    int32_t m = 0;
    for (int w = 0; w < kWarps; ++w) m += sm[w];
    a.part_m[b] = m;
  }
}

// Adds the blocks' partials in block order: one block, one thread per expert.
__global__ void __launch_bounds__(1024) rc_gate_stats_kernel(const __grid_constant__ GateParams a) {
  __shared__ float red[32];
  __shared__ int64_t tot[32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t m = 0;
  for (int b = threadIdx.x; b < a.p * a.blocks; b += blockDim.x) m += a.part_m[b];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m += __shfl_xor_sync(0xffffffffu, m, d);
  if (lane == 0) tot[warp] = m;
  __syncthreads();
  m = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) m += tot[w];
  const float M = (float)m, inv = 1.0f / fmaxf(M, 1.0f);
  float dot = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float s = 0.0f;
    int64_t c = 0;
    for (int r = 0; r < a.p; ++r) {
      int32_t cr = 0;
      for (int b = 0; b < a.blocks; ++b) {
        const uint64_t at = ((uint64_t)r * a.blocks + b) * a.E + e;
        s += a.part_p[at];
        cr += a.part_c[at];
      }
      a.counts[r][e] = cr;
      c += cr;
    }
    const float f = (float)c / ((float)a.k * fmaxf(M, 1.0f)), mean = s * inv;
    a.stats[e] = f;
    a.stats[a.E + e] = mean;
    dot += f * mean;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if (lane == 0) red[warp] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) s += red[w];
    a.stats[2 * a.E] = M;
    a.loss[0] = a.coef * (float)a.E * s;
  }
}

// dz of one token: with a_e = dloss * coef * E * f_e / M, S = the chosen
// experts' probabilities, and q_i = p_i / S (normalised) or p_i:
//   dz = p (a - sum p a) + [chosen] q dw - (normalised: [chosen] q, else p) * sum_i q_i dw_i
template <class T, int LPT, int VPL>
__global__ void __launch_bounds__(kNT) rc_gate_backward_kernel(const __grid_constant__ GateParams a) {
  constexpr int TPW = 32 / LPT;
  constexpr int V = kVec<T>;
  pdl_wait();
  const int r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (LPT - 1), e0 = sub * VPL;
  const float M = a.stats[2 * a.E];
  const float c = a.dloss ? a.dloss[0] * a.coef * (float)a.E / fmaxf(M, 1.0f) : 0.0f;
  float slope[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) slope[j] = e0 + j < a.E ? c * a.stats[e0 + j] : 0.0f;
  const uint64_t step = (uint64_t)gridDim.x * kWarps * TPW;
  for (uint64_t t0 = ((uint64_t)blockIdx.x * kWarps + warp) * TPW; t0 < a.tokens; t0 += step) {
    const uint64_t t = t0 + lane / LPT;
    const bool have = t < a.tokens;
    const bool unmasked = have && (a.mask[r] == nullptr || a.mask[r][t] != 0);
    const char *row = a.z[r] + t * (uint64_t)a.E * T::kBytes;
    float z[VPL], p[VPL], g[VPL];
    uint32_t sel = 0;
    if (unmasked) {
      load_row<T, VPL>(row, e0, a.E, a.vec, z);
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) z[j] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) g[j] = 0.0f;
    if (unmasked && a.dw[r]) {
      for (int i = 0; i < a.k; ++i) {
        const int id = a.ids[r][t * a.k + i];
        const float d = a.dw[r][t * a.k + i];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          if (id == e0 + j) {
            sel |= 1u << j;
            g[j] = d;
          }
        }
      }
    }
    bool live;
    const float total = row_exp<LPT, VPL>(z, p, &live);
    const float inv = live ? 1.0f / total : 0.0f;
    float pa = 0.0f, ps = 0.0f, pd = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      p[j] *= inv;
      pa += p[j] * slope[j];
      ps += (sel >> j) & 1u ? p[j] : 0.0f;
      pd += p[j] * g[j];
    }
    pa = row_sum<LPT>(pa);
    ps = row_sum<LPT>(ps);
    pd = row_sum<LPT>(pd);
    const float q = a.norm ? (ps > 0.0f ? 1.0f / ps : 0.0f) : 1.0f;
    const float inner = pd * q;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const bool s = (sel >> j) & 1u;
      float d = p[j] * (slope[j] - pa);
      if (a.norm) {
        if (s) d += p[j] * q * (g[j] - inner);
      } else {
        d += p[j] * ((s ? g[j] : 0.0f) - inner);
      }
      z[j] = live ? d : 0.0f;
    }
    if (!have) continue;
    char *out = a.dz[r] + t * (uint64_t)a.E * T::kBytes;
    if (a.vec) {
#pragma unroll
      for (int j = 0; j < VPL; j += V) {
        if (e0 + j < a.E) {
          float o[V];
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = z[j + i];
          store_vec<T, V>(out + (uint64_t)(e0 + j) * T::kBytes, o);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (e0 + j < a.E) store_elem<T>(out, e0 + j, z[j]);
    }
  }
}

// Blocks per rank: enough for the machine, at most one step of tokens each.
int blocks_per_rank(uint64_t tokens, int tpw, int p) {
  const uint64_t want = (tokens + (uint64_t)kWarps * tpw - 1) / ((uint64_t)kWarps * tpw);
  const uint64_t most = std::max(1, device_sm_count() * 2 / p);
  return (int)std::max<uint64_t>(1, std::min(want, most));
}

template <class T, int LPT, int VPL>
cudaError_t run(const GateJob &job, GateParams &a, cudaStream_t s) {
  cudaError_t err;
  if (job.backward) {
    const int blocks = blocks_per_rank(job.tokens, 32 / LPT, std::max(1, job.p / 4));
    return launch_kernel(rc_gate_backward_kernel<T, LPT, VPL>, dim3(blocks, job.p), dim3(kNT), 0, s, a);
  }
  a.blocks = blocks_per_rank(job.tokens, 32 / LPT, job.p);
  if (a.blocks > gate_max_blocks(job.p)) return cudaErrorInvalidValue;
  if ((err = launch_kernel(rc_gate_kernel<T, LPT, VPL>, dim3(a.blocks, job.p), dim3(kNT), 0, s, a)) != cudaSuccess)
    return err;
  const int nt = std::min(1024, (job.experts + 31) / 32 * 32);
  return launch_kernel(rc_gate_stats_kernel, dim3(1), dim3(nt), 0, s, a);
}

// Lanes per token: the fewest that hold the row at 8 values each, so that
// short rows share a warp; 16 values beyond 256 experts.
template <class T>
cudaError_t by_experts(const GateJob &job, GateParams &a, cudaStream_t s) {
  const int E = job.experts;
  if (E <= 8) return run<T, 1, 8>(job, a, s);
  if (E <= 16) return run<T, 2, 8>(job, a, s);
  if (E <= 32) return run<T, 4, 8>(job, a, s);
  if (E <= 64) return run<T, 8, 8>(job, a, s);
  if (E <= 128) return run<T, 16, 8>(job, a, s);
  if (E <= 256) return run<T, 32, 8>(job, a, s);
  return run<T, 32, 16>(job, a, s);
}

}  // namespace

int gate_max_blocks(int p) { return std::max(1, device_sm_count() * 2 / p); }

cudaError_t launch_gate(const GateJob &job, cudaStream_t s) {
  GateParams a{};
  const int esz = job.dt == kBF16 ? 2 : 4;
  uintptr_t all = 0;
  for (int r = 0; r < job.p; ++r) {
    a.z[r] = static_cast<const char *>(job.logits[r]);
    a.mask[r] = job.mask[r];
    a.ids[r] = job.ids[r];
    a.w[r] = job.weights[r];
    a.counts[r] = job.counts[r];
    a.dw[r] = job.dweights[r];
    a.dz[r] = static_cast<char *>(job.dlogits[r]);
    all |= reinterpret_cast<uintptr_t>(job.logits[r]) | reinterpret_cast<uintptr_t>(job.dlogits[r]);
  }
  a.vec = all % 16 == 0 && (job.experts * esz) % 16 == 0;
  a.stats = job.stats;
  a.loss = job.loss;
  a.dloss = job.dloss;
  a.tokens = job.tokens;
  a.E = job.experts;
  a.k = job.top_k;
  a.p = job.p;
  a.coef = job.coef;
  a.norm = job.normalize;
  if (!job.backward) {
    const uint64_t rows = (uint64_t)gate_max_blocks(job.p) * job.p;
    a.part_p = static_cast<float *>(job.ws);
    a.part_c = reinterpret_cast<int32_t *>(a.part_p + rows * job.experts);
    a.part_m = a.part_c + rows * job.experts;
  }
  if (job.dt == kF32) return by_experts<F32>(job, a, s);
  if (job.dt == kBF16) return by_experts<BF16>(job, a, s);
  return cudaErrorInvalidValue;
}

size_t gate_workspace(int p, int experts) {
  return (size_t)gate_max_blocks(p) * p * ((size_t)experts * 8 + 4);
}

}  // namespace rc

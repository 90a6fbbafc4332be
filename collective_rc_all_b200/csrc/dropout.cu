// dropout.cu -- dropout from a counter-based generator, alone over p rank
// buffers and behind a flat all-reduce, with an optional residual add.
//
// The mask is a function of the element's index, so it is never stored: the
// backward pass is the same call on the gradient.  Element e of the index
// space uses half word e % 8 of the Philox4x32-10 block with counter
// (e / 8, 0) and key `seed` (Salmon, Moraes, Dror, Shaw: "Parallel random
// numbers: as easy as 1, 2, 3", SC'11: ten rounds of two 32x32 -> 64-bit
// products, the key advanced by two Weyl constants).  The element is kept
// when the half word is at least t, and multiplied by `factor` =
// scale / (1 - t / 2^16), so the expectation is exact for the probability
// that is drawn (prob rounded to a multiple of 2^-16).
//
// 16 bits per element, not 32: a 16-byte bf16 vector then costs one Philox
// block (about 80 integer instructions for 8 elements), which stays under the
// time that its bytes take; with 32 bits per element the generator would need
// more issue slots than the memory leaves.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace rc {
namespace {

constexpr int kNT = 256;

struct DropParams {
  const char *x[kMaxRanks];
  const char *res[kMaxRanks];  // residuals (when the kernel adds them)
  char *y[kMaxRanks];
  uint64_t first[kMaxRanks];  // index of element 0 of each rank's buffer
  uint64_t n;
  uint64_t C;  // all-reduce: chunk length ceil(n/p)
  uint32_t k0, k1;
  uint32_t thr;  // keep when the half word >= thr; 65536 drops everything
  float factor;  // scale / (1 - thr / 2^16)
  int p;
};

// Bit j: element 8 * block + j is kept.
__device__ __forceinline__ uint32_t keep8(uint64_t block, uint32_t k0, uint32_t k1, uint32_t thr) {
  uint32_t a = (uint32_t)block, b = (uint32_t)(block >> 32), c = 0, d = 0;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t u = (uint64_t)a * 0xD2511F53u;
    const uint64_t v = (uint64_t)c * 0xCD9E8D57u;
    a = (uint32_t)(v >> 32) ^ b ^ k0;
    c = (uint32_t)(u >> 32) ^ d ^ k1;
    b = (uint32_t)v;
    d = (uint32_t)u;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  const uint32_t w[4] = {a, b, c, d};
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m |= (w[j] & 0xffffu) >= thr ? 1u << (2 * j) : 0u;
    m |= (w[j] >> 16) >= thr ? 2u << (2 * j) : 0u;
  }
  return m;
}

// Bit j: element e + j is kept, j < VEC <= 8.  A run that starts inside a
// block may need the next block too (e + 8 wraps with the index); the branch is the same for every vector
// of a buffer whose first index is a multiple of VEC.
template <int VEC>
__device__ __forceinline__ uint32_t keep_run(uint64_t e, const DropParams &a) {
  const uint32_t lane = (uint32_t)e & 7u;
  uint32_t m = keep8(e >> 3, a.k0, a.k1, a.thr);
  if (lane + VEC > 8) m |= keep8((e + 8) >> 3, a.k0, a.k1, a.thr) << 8;
  return m >> lane;
}

// A dropped element is a select, not a product: whatever it held (infinities
// and NaN too) becomes zero.
__device__ __forceinline__ float drop(float v, bool kept, float factor) {
  return kept ? __fmul_rn(v, factor) : 0.0f;
}

// Elements [e0, e1) of one rank, one at a time.
template <class T, bool RES>
__device__ __forceinline__ void drop_scalar(const DropParams &a, int r, uint64_t e0, uint64_t e1, uint64_t step) {
  for (uint64_t e = e0; e < e1; e += step) {
    const bool kept = keep_run<1>(a.first[r] + e, a) & 1u;
    float v = drop(load_elem<T>(a.x[r], e), kept, a.factor);
    if constexpr (RES) v = __fadd_rn(load_elem<T>(a.res[r], e), v);
    store_elem<T>(a.y[r], e, v);
  }
}

// 32 bytes of a buffer at a 32-byte boundary, streaming (see ld_stream_v4 and
// st_v4_cs).
struct Raw32 {
  uint4 lo, hi;
};
__device__ __forceinline__ Raw32 ld_stream_32(const void *p) {
  Raw32 r;
  asm("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r.lo.x), "=r"(r.lo.y), "=r"(r.lo.z), "=r"(r.lo.w), "=r"(r.hi.x), "=r"(r.hi.y), "=r"(r.hi.z),
        "=r"(r.hi.w)
      : "l"(p));
  return r;
}
__device__ __forceinline__ void st_cs_32(void *p, const Raw32 &r) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.lo.x), "r"(r.lo.y), "r"(r.lo.z),
               "r"(r.lo.w), "r"(r.hi.x), "r"(r.hi.y), "r"(r.hi.z), "r"(r.hi.w)
               : "memory");
}

// One vector: dropped by the low bits of m, added to the residual's, packed.
template <class T, bool RES>
__device__ __forceinline__ uint4 drop_vec(const uint4 &x, const uint4 &res, uint32_t m, float factor) {
  constexpr int VEC = kVec<T>;
  float f[VEC];
  unpack<T>(x, f);
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] = drop(f[j], (m >> j) & 1u, factor);
  if constexpr (RES) {
    float g[VEC];
    unpack<T>(res, g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = __fadd_rn(g[j], f[j]);
  }
  if constexpr (std::is_same<T, BF16>::value) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  } else {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
}

// One thread per BYTES of one rank (32, or 16 where a buffer is aligned to no
// more); the thread after the last whole piece takes the tail.  32 bytes are
// one Philox block's 8 elements in fp32 and two blocks in bf16, and twice the
// bytes in flight: 8 x 2,097,152 fp32 29.5 -> 18.3 us, 8 x 16,777,216 bf16 with
// residual 137 -> 118 us.
template <class T, bool RES, int BYTES>
__global__ void __launch_bounds__(kNT) rc_dropout_kernel(const __grid_constant__ DropParams a) {
  pdl_wait();
  constexpr int VEC = kVec<T>, N = VEC * BYTES / 16;
  const int r = blockIdx.y;
  const uint64_t v = (uint64_t)blockIdx.x * kNT + threadIdx.x;
  const uint64_t e = v * N;
  if (e >= a.n) return;
  if (e + N > a.n) {
    drop_scalar<T, RES>(a, r, e, a.n, 1);
    return;
  }
  if constexpr (BYTES == 32) {
    const Raw32 x = ld_stream_32(a.x[r] + v * 32);
    Raw32 g{};
    if constexpr (RES) g = ld_stream_32(a.res[r] + v * 32);
    uint32_t lo, hi;
    if constexpr (N == 8) {
      lo = keep_run<8>(a.first[r] + e, a);
      hi = lo >> VEC;
    } else {
      lo = keep_run<8>(a.first[r] + e, a);
      hi = keep_run<8>(a.first[r] + e + 8, a);
    }
    Raw32 y;
    y.lo = drop_vec<T, RES>(x.lo, g.lo, lo, a.factor);
    y.hi = drop_vec<T, RES>(x.hi, g.hi, hi, a.factor);
    st_cs_32(a.y[r] + v * 32, y);
  } else {
    const uint4 x = ld_stream_v4(a.x[r] + v * 16);
    uint4 g = make_uint4(0, 0, 0, 0);
    if constexpr (RES) g = ld_stream_v4(a.res[r] + v * 16);
    st_v4_cs(a.y[r] + v * 16, drop_vec<T, RES>(x, g, keep_run<VEC>(a.first[r] + e, a), a.factor));
  }
}

// Buffers that are not 16-byte aligned.
template <class T, bool RES>
__global__ void __launch_bounds__(kNT) rc_dropout_scalar_kernel(const __grid_constant__ DropParams a) {
  pdl_wait();
  drop_scalar<T, RES>(a, blockIdx.y, (uint64_t)blockIdx.x * kNT + threadIdx.x, a.n, (uint64_t)gridDim.x * kNT);
}

__device__ __forceinline__ int ring_rank(int c, int k, int p) {
  const int r = c + 1 + k;
  return r >= p ? r - p : r;
}

// The all-reduce's fold of one element (ring order of its chunk), dropped,
// added to every rank's residual and stored to every rank.
template <class T, bool RES>
__device__ __forceinline__ void reduce_drop_elem(const DropParams &a, uint64_t e) {
  const int c = (int)(e / a.C);
  float acc = load_elem<T>(a.x[ring_rank(c, 0, a.p)], e);
  for (int k = 1; k < a.p; ++k) acc = combine<kSum>(acc, load_elem<T>(a.x[ring_rank(c, k, a.p)], e));
  const float v = drop(acc, keep_run<1>(a.first[0] + e, a) & 1u, a.factor);
  for (int r = 0; r < a.p; ++r)
    store_elem<T>(a.y[r], e, RES ? __fadd_rn(load_elem<T>(a.res[r], e), v) : v);
}

// One thread per 16-byte vector: p loads in flight, the fold, one mask for all
// ranks (a replicated activation), p residual adds and p stores.  A vector
// that straddles a chunk border, whose elements fold in two orders, and the
// tail go element by element.
template <int PMAX, class T, bool RES>
__global__ void __launch_bounds__(kNT) rc_reduce_dropout_kernel(const __grid_constant__ DropParams a) {
  pdl_wait();
  constexpr int VEC = kVec<T>;
  const int p = a.p;
  const uint64_t v = (uint64_t)blockIdx.x * kNT + threadIdx.x;
  const uint64_t e = v * VEC;
  if (e >= a.n) return;
  // the block's first chunk by division, the thread's by stepping from there
  const uint64_t eb = (uint64_t)blockIdx.x * kNT * VEC;
  uint64_t c = eb / a.C;
  uint64_t cend = (c + 1) * a.C;
  while (e >= cend) {
    ++c;
    cend += a.C;
  }
  if (e + VEC > a.n || e + VEC > cend) {
    const uint64_t end = e + VEC < a.n ? e + VEC : a.n;
    for (uint64_t i = e; i < end; ++i) reduce_drop_elem<T, RES>(a, i);
    return;
  }
  uint4 raw[PMAX], rr[PMAX];
#pragma unroll
  for (int k = 0; k < PMAX; ++k)
    if (k < p) raw[k] = ld_stream_v4(a.x[ring_rank((int)c, k, p)] + v * 16);
  if constexpr (RES) {
#pragma unroll
    for (int k = 0; k < PMAX; ++k)
      if (k < p) rr[k] = ld_stream_v4(a.res[k] + v * 16);
  }
  const uint32_t m = keep_run<VEC>(a.first[0] + e, a);
  float acc[VEC];
  unpack<T>(raw[0], acc);
#pragma unroll
  for (int k = 1; k < PMAX; ++k) {
    if (k < p) {
      float w[VEC];
      unpack<T>(raw[k], w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] = combine<kSum>(acc[j], w[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = drop(acc[j], (m >> j) & 1u, a.factor);
#pragma unroll
  for (int k = 0; k < PMAX; ++k) {
    if (k < p) {
      if constexpr (RES) {
        float w[VEC];
        unpack<T>(rr[k], w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = __fadd_rn(w[j], acc[j]);
        store_vec<T, VEC, true>(a.y[k] + v * 16, w);
      } else {
        store_vec<T, VEC, true>(a.y[k] + v * 16, acc);
      }
    }
  }
}

template <class T, bool RES>
__global__ void __launch_bounds__(kNT) rc_reduce_dropout_scalar_kernel(const __grid_constant__ DropParams a) {
  pdl_wait();
  for (uint64_t e = (uint64_t)blockIdx.x * kNT + threadIdx.x; e < a.n; e += (uint64_t)gridDim.x * kNT)
    reduce_drop_elem<T, RES>(a, e);
}

template <class T, bool RES>
cudaError_t run(const DropoutJob &job, cudaStream_t s) {
  DropParams a{};
  const int p = job.p;
  uintptr_t all = 0;
  for (int r = 0; r < p; ++r) {
    a.x[r] = static_cast<const char *>(job.x[r]);
    a.res[r] = static_cast<const char *>(job.res[r]);
    a.y[r] = static_cast<char *>(job.y[r]);
    a.first[r] = job.offset + (uint64_t)r * job.rank_stride;
    all |= reinterpret_cast<uintptr_t>(job.x[r]) | reinterpret_cast<uintptr_t>(job.res[r]) |
           reinterpret_cast<uintptr_t>(job.y[r]);
  }
  a.n = job.n;
  a.C = (job.n + p - 1) / p;
  a.k0 = (uint32_t)job.seed;
  a.k1 = (uint32_t)(job.seed >> 32);
  a.thr = job.thr;
  a.factor = job.factor;
  a.p = p;
  const uint64_t vec_blocks = ((job.n + kVec<T> - 1) / kVec<T> + kNT - 1) / kNT;
  const uint64_t elem_blocks = std::min<uint64_t>((job.n + kNT - 1) / kNT, (uint64_t)device_sm_count() * 8);
  if (vec_blocks > 0x7fffffffull) return cudaErrorInvalidValue;
  const bool aligned = all % 16 == 0;
  if (!job.reduce) {
    if (all % 32 == 0)
      return launch_kernel(rc_dropout_kernel<T, RES, 32>, dim3((unsigned)((vec_blocks + 1) / 2), p), dim3(kNT), 0, s,
                           a);
    if (aligned)
      return launch_kernel(rc_dropout_kernel<T, RES, 16>, dim3((unsigned)vec_blocks, p), dim3(kNT), 0, s, a);
    return launch_kernel(rc_dropout_scalar_kernel<T, RES>, dim3((unsigned)elem_blocks, p), dim3(kNT), 0, s, a);
  }
  if (!aligned)
    return launch_kernel(rc_reduce_dropout_scalar_kernel<T, RES>, dim3((unsigned)elem_blocks), dim3(kNT), 0, s, a);
  const dim3 grid((unsigned)vec_blocks);
  if (p <= 2) return launch_kernel(rc_reduce_dropout_kernel<2, T, RES>, grid, dim3(kNT), 0, s, a);
  if (p <= 4) return launch_kernel(rc_reduce_dropout_kernel<4, T, RES>, grid, dim3(kNT), 0, s, a);
  if (p <= 8) return launch_kernel(rc_reduce_dropout_kernel<8, T, RES>, grid, dim3(kNT), 0, s, a);
  return launch_kernel(rc_reduce_dropout_kernel<16, T, RES>, grid, dim3(kNT), 0, s, a);
}

}  // namespace

cudaError_t launch_dropout(const DropoutJob &job, cudaStream_t s) {
  const bool res = job.res[0] != nullptr;
  if (job.dt == kF32) return res ? run<F32, true>(job, s) : run<F32, false>(job, s);
  if (job.dt == kBF16) return res ? run<BF16, true>(job, s) : run<BF16, false>(job, s);
  return cudaErrorInvalidValue;
}

}  // namespace rc

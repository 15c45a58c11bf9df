// gradclip.cu -- the norm over every gradient of a model, and gradients
// scaled by it (clipping).
//
//   N = (sum_i sum_e |g_i[e]|^p)^(1/p)      p = 1, 2, or the largest |g| (inf)
//   s = min(1, max_norm / (N + eps))
//   out_i[e] = round(fp32(s * g_i[e]))      in place or into other tensors
//
// Two launches: grad_partial_kernel reads every gradient once and leaves one
// partial sum per CTA in the caller's workspace; the second launch sums the
// partials, each of its CTAs for itself and in one fixed order, and either
// writes N and s (grad_finish_kernel) or scales the gradients
// (grad_scale_kernel).  Nothing is counted or accumulated with atomics: the
// same call on the same device gives the same bits.
//
// The squares are formed and summed in fp64.  In fp32 a square underflows
// below |g| ~ 1e-19 and overflows above 1.8e19; in fp64 neither happens for
// any fp32 input, the square is exact, and a sum of 2^40 of them is good to
// far below the one rounding of N to fp32.  The maximum is taken over the bit
// patterns of |g| as integers, which order like the values and place every
// NaN above infinity, so a NaN is never lost.
#include "internal.h"

#include <cuda_fp16.h>

namespace muon {
namespace {

// ---------------------------------------------------------------- element types
template <int DT>
struct Elem;
template <>
struct Elem<MUON_F32> {
  typedef float T;
  static constexpr int E = 4;                       // elements of a 16-byte vector
  static __device__ __forceinline__ void unpack(const uint4& r, float* f) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ float widen(float x) { return x; }
  static __device__ __forceinline__ float narrow(float x) { return x; }
};
template <>
struct Elem<MUON_BF16> {
  typedef __nv_bfloat16 T;
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<MUON_F16> {
  typedef __half T;
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[k]);
      f[2 * k] = __low2float(h);
      f[2 * k + 1] = __high2float(h);
    }
  }
  static __device__ __forceinline__ float widen(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }
};

// ---------------------------------------------------------------- sums
// One running value of a norm.  Sums are doubles; the maximum is the bit
// pattern of |g|, held in the same 8-byte word.
template <int P>
struct Acc {
  double v = 0.0;
  __device__ __forceinline__ void add(float g) {
    const double d = (double)g;
    if (P == GRAD_L2) v = fma(d, d, v);
    else v += fabs(d);
  }
  __device__ __forceinline__ void join(const Acc& o) { v += o.v; }
  __device__ __forceinline__ Acc shuffled(int mask) const {
    Acc o;
    o.v = __shfl_xor_sync(0xffffffffu, v, mask);
    return o;
  }
  __device__ __forceinline__ unsigned long long word() const { return __double_as_longlong(v); }
  __device__ __forceinline__ void set(unsigned long long w) { v = __longlong_as_double(w); }
  __device__ __forceinline__ double norm() const { return P == GRAD_L2 ? sqrt(v) : v; }
};
template <>
struct Acc<GRAD_INF> {
  unsigned v = 0;
  __device__ __forceinline__ void add(float g) { v = max(v, __float_as_uint(g) & 0x7fffffffu); }
  __device__ __forceinline__ void join(const Acc& o) { v = max(v, o.v); }
  __device__ __forceinline__ Acc shuffled(int mask) const {
    Acc o;
    o.v = __shfl_xor_sync(0xffffffffu, v, mask);
    return o;
  }
  __device__ __forceinline__ unsigned long long word() const { return v; }
  __device__ __forceinline__ void set(unsigned long long w) { v = (unsigned)w; }
  __device__ __forceinline__ double norm() const { return (double)__uint_as_float(v); }
};

// Joins the CTA's values in a fixed order; every thread gets the result.
template <int P>
__device__ __forceinline__ Acc<P> block_join(Acc<P> a, unsigned long long* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a.join(a.shuffled(o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a.word();
  __syncthreads();
  Acc<P> t;
#pragma unroll
  for (int w = 0; w < GRAD_THREADS / 32; ++w) {
    Acc<P> x;
    x.set(red[w]);
    t.join(x);
  }
  __syncthreads();   // red may be written again
  return t;
}

// ---------------------------------------------------------------- tensors as 16-byte vectors
// A tensor whose first element lies `mis` elements past a 16-byte boundary is
// walked in the aligned vectors that cover it: vector v holds elements
// [v E - mis, (v + 1) E - mis).  Only the first and the last can be partial;
// those are read element by element, so nothing outside the tensor is touched.
template <int P, int DT>
__device__ __forceinline__ void partial_chunk(const GradTensor& T, long long v0, Acc<P>& acc) {
  typedef Elem<DT> X;
  constexpr int E = X::E;
  const typename X::T* g = reinterpret_cast<const typename X::T*>(T.g);
  const long long nvec = (T.numel + T.mis + E - 1) / E;
  uint4 raw[GRAD_VEC];
  bool full[GRAD_VEC];
#pragma unroll
  for (int j = 0; j < GRAD_VEC; ++j) {
    const long long v = v0 + threadIdx.x + j * GRAD_THREADS;
    const long long e = v * E - T.mis;
    full[j] = e >= 0 && e + E <= T.numel;
    raw[j] = make_uint4(0, 0, 0, 0);
    if (full[j]) raw[j] = __ldg(reinterpret_cast<const uint4*>(g + e));
  }
#pragma unroll
  for (int j = 0; j < GRAD_VEC; ++j) {
    const long long v = v0 + threadIdx.x + j * GRAD_THREADS;
    if (full[j]) {
      float f[E];
      X::unpack(raw[j], f);
#pragma unroll
      for (int k = 0; k < E; ++k) acc.add(f[k]);
    } else if (v < nvec) {
      const long long e = v * E - T.mis;
      for (int k = 0; k < E; ++k)
        if (e + k >= 0 && e + k < T.numel) acc.add(X::widen(g[e + k]));
    }
  }
}

template <int P>
__global__ void __launch_bounds__(GRAD_THREADS) grad_partial_kernel(const __grid_constant__ GradLaunch L) {
  __shared__ unsigned long long red[GRAD_THREADS / 32];
  Acc<P> acc;
  int ti = 0;
  for (int c = blockIdx.x; c < L.nchunks; c += gridDim.x) {
    while (ti + 1 < L.n && L.t[ti + 1].chunk0 <= c) ++ti;   // chunks only grow
    const GradTensor& T = L.t[ti];
    const long long v0 = (long long)(c - T.chunk0) * GRAD_CHUNK_VECS;
    if (T.dtype == MUON_F32) partial_chunk<P, MUON_F32>(T, v0, acc);
    else if (T.dtype == MUON_BF16) partial_chunk<P, MUON_BF16>(T, v0, acc);
    else partial_chunk<P, MUON_F16>(T, v0, acc);
  }
  acc = block_join<P>(acc, red);
  if (threadIdx.x == 0) L.partials[L.part0 + blockIdx.x] = acc.word();
}

// N and s from the partials, the same in every thread of every CTA that asks.
// s is formed in fp64 from the unrounded N; a NaN norm gives a NaN scale.
template <int P>
__device__ __forceinline__ float finish(const GradLaunch& L, unsigned long long* red, float* norm) {
  Acc<P> acc;
  for (int i = threadIdx.x; i < L.npartials; i += GRAD_THREADS) {
    Acc<P> x;
    x.set(__ldcg(L.partials + i));
    acc.join(x);
  }
  const double nrm = block_join<P>(acc, red).norm();
  *norm = (float)nrm;
  const double den = nrm + L.eps;
  const double s = (isinf(L.max_norm) || den == 0.0) ? 1.0 : L.max_norm / den;
  return s >= 1.0 ? 1.f : (float)s;
}

template <int P>
__global__ void __launch_bounds__(GRAD_THREADS) grad_finish_kernel(const __grid_constant__ GradLaunch L) {
  __shared__ unsigned long long red[GRAD_THREADS / 32];
  float norm;
  const float s = finish<P>(L, red, &norm);
  if (threadIdx.x == 0) {
    *L.norm = norm;
    if (L.scale) *L.scale = s;
  }
}

template <int DT, int OT>
__device__ __forceinline__ void scale_chunk(const GradTensor& T, long long v0, float s) {
  typedef Elem<DT> X;
  typedef Elem<OT> Y;
  constexpr int E = X::E;
  const typename X::T* g = reinterpret_cast<const typename X::T*>(T.g);
  typename Y::T* out = reinterpret_cast<typename Y::T*>(T.out);
  const long long nvec = (T.numel + T.mis + E - 1) / E;
  uint4 raw[GRAD_VEC];
  bool full[GRAD_VEC];
#pragma unroll
  for (int j = 0; j < GRAD_VEC; ++j) {
    const long long v = v0 + threadIdx.x + j * GRAD_THREADS;
    const long long e = v * E - T.mis;
    full[j] = e >= 0 && e + E <= T.numel;
    raw[j] = make_uint4(0, 0, 0, 0);
    if (full[j]) raw[j] = *reinterpret_cast<const uint4*>(g + e);
  }
#pragma unroll
  for (int j = 0; j < GRAD_VEC; ++j) {
    const long long v = v0 + threadIdx.x + j * GRAD_THREADS;
    const long long e = v * E - T.mis;
    if (full[j]) {
      float f[E];
      X::unpack(raw[j], f);
      union {
        typename Y::T y[E];
        uint4 q[sizeof(typename Y::T) * E / 16 > 0 ? sizeof(typename Y::T) * E / 16 : 1];
        uint2 d;
      } o;
#pragma unroll
      for (int k = 0; k < E; ++k) o.y[k] = Y::narrow(__fmul_rn(s, f[k]));
      if (T.out_vec) {
        if constexpr (sizeof(typename Y::T) * E >= 16) {
#pragma unroll
          for (int q = 0; q < (int)sizeof(typename Y::T) * E / 16; ++q)
            reinterpret_cast<uint4*>(out + e)[q] = o.q[q];
        } else {
          *reinterpret_cast<uint2*>(out + e) = o.d;
        }
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k) out[e + k] = o.y[k];
      }
    } else if (v < nvec) {
      for (int k = 0; k < E; ++k)
        if (e + k >= 0 && e + k < T.numel)
          out[e + k] = Y::narrow(__fmul_rn(s, X::widen(g[e + k])));
    }
  }
}

template <int DT>
__device__ __forceinline__ void scale_chunk_to(const GradTensor& T, long long v0, float s) {
  if (T.out_dtype == MUON_F32) scale_chunk<DT, MUON_F32>(T, v0, s);
  else if (T.out_dtype == MUON_BF16) scale_chunk<DT, MUON_BF16>(T, v0, s);
  else scale_chunk<DT, MUON_F16>(T, v0, s);
}

template <int P>
__global__ void __launch_bounds__(GRAD_THREADS) grad_scale_kernel(const __grid_constant__ GradLaunch L) {
  __shared__ unsigned long long red[GRAD_THREADS / 32];
  float norm;
  const float s = finish<P>(L, red, &norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (L.norm) *L.norm = norm;
    if (L.scale) *L.scale = s;
  }
  int ti = 0;
  for (int c = blockIdx.x; c < L.nchunks; c += gridDim.x) {
    while (ti + 1 < L.n && L.t[ti + 1].chunk0 <= c) ++ti;
    const GradTensor& T = L.t[ti];
    if (s == 1.f && T.out == T.g) continue;   // in place and under the bound: 1 * g is g
    const long long v0 = (long long)(c - T.chunk0) * GRAD_CHUNK_VECS;
    if (T.dtype == MUON_F32) scale_chunk_to<MUON_F32>(T, v0, s);
    else if (T.dtype == MUON_BF16) scale_chunk_to<MUON_BF16>(T, v0, s);
    else scale_chunk_to<MUON_F16>(T, v0, s);
  }
}

template <int P>
cudaError_t launch(const GradLaunch& L, GradStage stage, int grid, cudaStream_t stream) {
  if (stage == GRAD_STAGE_PARTIAL) grad_partial_kernel<P><<<grid, GRAD_THREADS, 0, stream>>>(L);
  else if (stage == GRAD_STAGE_FINISH) grad_finish_kernel<P><<<1, GRAD_THREADS, 0, stream>>>(L);
  else grad_scale_kernel<P><<<grid, GRAD_THREADS, 0, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace

int grad_blocks_per_sm() {
  int a = 0, b = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&a, grad_partial_kernel<GRAD_L2>, GRAD_THREADS, 0) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, grad_scale_kernel<GRAD_L2>, GRAD_THREADS, 0) !=
          cudaSuccess)
    return 1;
  const int n = a < b ? a : b;
  return n < 1 ? 1 : n;
}

cudaError_t launch_grad(const GradLaunch& L, int norm, GradStage stage, int grid, cudaStream_t stream) {
  if (norm == GRAD_L1) return launch<GRAD_L1>(L, stage, grid, stream);
  if (norm == GRAD_L2) return launch<GRAD_L2>(L, stage, grid, stream);
  return launch<GRAD_INF>(L, stage, grid, stream);
}

}  // namespace muon

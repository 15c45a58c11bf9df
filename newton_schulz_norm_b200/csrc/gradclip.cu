// gradclip.cu -- the norm over every gradient of a model, and gradients
// scaled by it (clipping).
//
//   N = (sum_i sum_e |g_i[e]|^p)^(1/p)      p = 1, 2, or the largest |g| (inf)
//   s = min(1, max_norm / (N + eps))
//   out_i[e] = round(fp32(s * g_i[e]))      in place or into other tensors
//
// Two forms, by the size of the list.  grad_cluster_kernel does all of it in
// one launch of one thread-block cluster, whose CTAs exchange their partial
// values through distributed shared memory.  Longer lists take two launches:
// grad_partial_kernel reads every gradient once and leaves one partial value
// per CTA in the caller's workspace; the second launch joins the partials,
// each of its CTAs for itself and in one fixed order, and either writes N and
// s (grad_finish_kernel) or scales the gradients (grad_scale_kernel).  The
// second launch is a programmatic dependent of the first: its CTAs are
// resident and waiting when the last partial value is written.  Nothing is
// counted or accumulated with atomics, and no workspace outlives the call:
// the same call on the same device gives the same bits, whatever runs beside.
//
// The squares are formed and summed in fp64.  In fp32 a square underflows
// below |g| ~ 1e-19 and overflows above 1.8e19; in fp64 neither happens for
// any fp32 input, the square is exact, and a sum of 2^40 of them is good to
// far below the one rounding of N to fp32.  The maximum is taken over the bit
// patterns of |g| as integers, which order like the values and place every
// NaN above infinity, so a NaN is never lost.
#include "internal.h"

#include <cooperative_groups.h>
#include <cuda_fp16.h>

namespace cg = cooperative_groups;

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
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
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
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
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

// Joins the values of THREADS threads in a fixed order; every thread gets the result.
template <int P, int THREADS>
__device__ __forceinline__ Acc<P> block_join(Acc<P> a, unsigned long long* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a.join(a.shuffled(o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a.word();
  __syncthreads();
  Acc<P> t;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
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
// Gradients are read with coherent loads only: in place, the scaling writes what
// the norm has read, in the same launch where one cluster does both.

// Whether chunk v0.. of the tensor is nothing but whole vectors.
__device__ __forceinline__ bool whole_chunk(const GradTensor& T, long long v0) {
  const int shift = T.dtype == MUON_F32 ? 2 : 3;   // log2 of a vector's elements
  return (v0 > 0 || T.mis == 0) && ((v0 + GRAD_CHUNK_VECS) << shift) <= T.numel + T.mis;
}

// The 16-byte boundary at or before the first element.
__device__ __forceinline__ const char* vector0(const GradTensor& T) {
  return reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(T.g) & ~(uintptr_t)15);
}

struct Raw {
  uint4 v[GRAD_VEC];
};

template <bool STREAMED>
__device__ __forceinline__ void load_chunk(const GradTensor& T, long long v0, int tid, Raw& r) {
  const uint4* p = reinterpret_cast<const uint4*>(vector0(T)) + v0 + tid;
#pragma unroll
  for (int j = 0; j < GRAD_VEC; ++j) r.v[j] = STREAMED ? __ldcs(p + j * GRAD_THREADS) : p[j * GRAD_THREADS];
}

template <int P, int DT>
__device__ __forceinline__ void add_vec(const uint4& v, Acc<P>& acc) {
  float f[Elem<DT>::E];
  Elem<DT>::unpack(v, f);
#pragma unroll
  for (int k = 0; k < Elem<DT>::E; ++k) acc.add(f[k]);
}

template <int P>
__device__ __forceinline__ void add_raw(const Raw& r, int dtype, Acc<P>& acc) {
#pragma unroll
  for (int j = 0; j < GRAD_VEC; ++j) {
    if (dtype == MUON_F32) add_vec<P, MUON_F32>(r.v[j], acc);
    else if (dtype == MUON_BF16) add_vec<P, MUON_BF16>(r.v[j], acc);
    else add_vec<P, MUON_F16>(r.v[j], acc);
  }
}

// A chunk with a partial vector, or the last one of a tensor.
template <int P, int DT>
__device__ __forceinline__ void add_ragged(const GradTensor& T, long long v0, int tid, Acc<P>& acc) {
  typedef Elem<DT> X;
  constexpr int E = X::E;
  const typename X::T* g = reinterpret_cast<const typename X::T*>(vector0(T));
  const long long end = T.numel + T.mis;   // elements are counted from vector 0 here
  const long long v1 = min(v0 + GRAD_CHUNK_VECS, (end + E - 1) / E);
#pragma unroll 4
  for (long long v = v0 + tid; v < v1; v += GRAD_THREADS) {
    const long long e = v * E;
    if (e >= T.mis && e + E <= end) {
      add_vec<P, DT>(*(reinterpret_cast<const uint4*>(g) + v), acc);
    } else {
      for (int k = 0; k < E; ++k)
        if (e + k >= T.mis && e + k < end) acc.add(X::widen(g[e + k]));
    }
  }
}

// Chunks c, c + step, ... below `end`; STREAMED: not to be kept in L2.
template <int P, bool STREAMED, int N>
__device__ __forceinline__ int add_chunks_to(const GradLaunch<N>& L, int c, int step, int end, int tid, int& ti,
                                             Acc<P>& acc) {
  for (; c < end; c += step) {
    ti = tensor_of(L.chunk0, L.n, c, ti);
    const GradTensor& T = L.t[ti];
    const long long v0 = (long long)(c - L.chunk0[ti]) * GRAD_CHUNK_VECS;
    if (whole_chunk(T, v0)) {
      Raw raw;
      load_chunk<STREAMED>(T, v0, tid, raw);
      add_raw<P>(raw, T.dtype, acc);
    } else if (T.dtype == MUON_F32) {
      add_ragged<P, MUON_F32>(T, v0, tid, acc);
    } else if (T.dtype == MUON_BF16) {
      add_ragged<P, MUON_BF16>(T, v0, tid, acc);
    } else {
      add_ragged<P, MUON_F16>(T, v0, tid, acc);
    }
  }
  return c;
}

// The norm's part of chunks first, first + step, ... of the launch.  Where the
// gradients are scaled afterwards, the chunks that the scaling reads first (the
// last ones) are left in L2 by passing the ones before through as streamed.  That
// is so for a list of one launch; the scaling of a longer one begins with the
// first launch's chunks, of which little is left by then.
template <int P, int N>
__device__ __forceinline__ Acc<P> add_chunks(const GradLaunch<N>& L, int first, int step, int tid) {
  Acc<P> acc;
  int ti = 0, c = first;
  if (L.scales) c = add_chunks_to<P, true>(L, c, step, L.nchunks - GRAD_KEEP_CHUNKS, tid, ti, acc);
  add_chunks_to<P, false>(L, c, step, L.nchunks, tid, ti, acc);
  return acc;
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <int P, int N>
__global__ void __launch_bounds__(GRAD_THREADS)
    grad_partial_kernel(const __grid_constant__ GradLaunch<N> L) {
  __shared__ unsigned long long red[GRAD_THREADS / 32];
  pdl_launch();
  const Acc<P> acc = block_join<P, GRAD_THREADS>(add_chunks<P>(L, blockIdx.x, gridDim.x, threadIdx.x), red);
  if (threadIdx.x == 0) L.h.partials[L.part0 + blockIdx.x] = acc.word();
}

// s from N, in fp64 and from the unrounded N.  A NaN norm gives a NaN scale
// whatever the bound; an infinite bound is never exceeded, not by an infinite
// norm either (s = 1), which a finite one turns into s = 0.
__device__ __forceinline__ float scale_of(double norm, const GradCall& h) {
  if (isnan(norm)) return (float)norm;
  const double den = norm + h.eps;
  const double s = (isinf(h.max_norm) || den == 0.0) ? 1.0 : h.max_norm / den;
  return s >= 1.0 ? 1.f : (float)s;
}

// N from the partials, the same in every thread of every CTA that asks.
template <int P>
__device__ __forceinline__ double joined(const GradCall& h, unsigned long long* red) {
  Acc<P> acc;
  for (int i = threadIdx.x; i < h.npartials; i += GRAD_THREADS) {
    Acc<P> x;
    x.set(__ldcg(h.partials + i));
    acc.join(x);
  }
  return block_join<P, GRAD_THREADS>(acc, red).norm();
}

__device__ __forceinline__ double joined(const GradCall& h, unsigned long long* red) {
  if (h.norm_kind == GRAD_L1) return joined<GRAD_L1>(h, red);
  if (h.norm_kind == GRAD_L2) return joined<GRAD_L2>(h, red);
  return joined<GRAD_INF>(h, red);
}

__device__ __forceinline__ void write_results(const GradCall& h, double norm, float s) {
  *h.norm = (float)norm;
  if (h.scale) *h.scale = s;
}

__global__ void __launch_bounds__(GRAD_THREADS) grad_finish_kernel(const __grid_constant__ GradCall h) {
  __shared__ unsigned long long red[GRAD_THREADS / 32];
  pdl_wait();
  const double norm = joined(h, red);
  if (threadIdx.x == 0) write_results(h, norm, scale_of(norm, h));
}

// ---------------------------------------------------------------- scaling
__device__ __forceinline__ void st32(void* p, const uint32_t* r) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Writes the E scaled elements of one vector.
template <int OT, int E>
__device__ __forceinline__ void store_vec(typename Elem<OT>::T* out, const float* f, float s, bool wide) {
  typedef Elem<OT> Y;
  constexpr int W = E * (int)sizeof(typename Y::T) / 4;   // words: 2, 4 or 8
  uint32_t w[W];
  if constexpr (OT == MUON_F32) {
#pragma unroll
    for (int k = 0; k < E; ++k) w[k] = __float_as_uint(__fmul_rn(s, f[k]));
  } else {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = Y::pack(__fmul_rn(s, f[2 * k]), __fmul_rn(s, f[2 * k + 1]));
  }
  if constexpr (W == 2) {
    __stcs(reinterpret_cast<uint2*>(out), make_uint2(w[0], w[1]));
  } else if constexpr (W == 4) {
    __stcs(reinterpret_cast<uint4*>(out), make_uint4(w[0], w[1], w[2], w[3]));
  } else {
    if (wide) {
      st32(out, w);
    } else {
      __stcs(reinterpret_cast<uint4*>(out), make_uint4(w[0], w[1], w[2], w[3]));
      __stcs(reinterpret_cast<uint4*>(out) + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
  }
}

// A whole chunk, already loaded, into an output that takes vectors.
template <int DT, int OT>
__device__ __forceinline__ void scale_raw(const GradTensor& T, long long v0, int tid, float s, const Raw& r) {
  constexpr int E = Elem<DT>::E;
  typename Elem<OT>::T* out = reinterpret_cast<typename Elem<OT>::T*>(T.out) - T.mis + (v0 + tid) * E;
#pragma unroll
  for (int j = 0; j < GRAD_VEC; ++j) {
    float f[E];
    Elem<DT>::unpack(r.v[j], f);
    store_vec<OT, E>(out + j * GRAD_THREADS * E, f, s, T.out_vec > 1);
  }
}

template <int DT, int OT>
__device__ __forceinline__ void scale_ragged(const GradTensor& T, long long v0, int tid, float s) {
  typedef Elem<DT> X;
  typedef Elem<OT> Y;
  constexpr int E = X::E;
  const typename X::T* g = reinterpret_cast<const typename X::T*>(vector0(T));
  typename Y::T* out = reinterpret_cast<typename Y::T*>(T.out) - T.mis;
  const long long end = T.numel + T.mis;   // elements are counted from vector 0 here
  if (T.out_vec) {
    const long long v1 = min(v0 + GRAD_CHUNK_VECS, (end + E - 1) / E);
    for (long long v = v0 + tid; v < v1; v += GRAD_THREADS) {
      const long long e = v * E;
      if (e >= T.mis && e + E <= end) {
        float f[E];
        X::unpack(*(reinterpret_cast<const uint4*>(g) + v), f);
        store_vec<OT, E>(out + e, f, s, T.out_vec > 1);
      } else {
        for (int k = 0; k < E; ++k)
          if (e + k >= T.mis && e + k < end) out[e + k] = Y::narrow(__fmul_rn(s, X::widen(g[e + k])));
      }
    }
    return;
  }
  // The output is not aligned where the input is: single elements, neighbours
  // in neighbouring threads.
  const long long e1 = min((v0 + GRAD_CHUNK_VECS) * E, end);
#pragma unroll 4
  for (long long e = max(v0 * E, (long long)T.mis) + tid; e < e1; e += GRAD_THREADS)
    out[e] = Y::narrow(__fmul_rn(s, X::widen(g[e])));
}

// One chunk; `raw` holds it already if `loaded` (then it is whole and its
// output takes vectors).
template <int DT, int OT>
__device__ __forceinline__ void scale_chunk(const GradTensor& T, long long v0, int tid, float s, bool loaded,
                                            Raw& raw) {
  if (!loaded) {
    if (!T.out_vec || !whole_chunk(T, v0)) {
      scale_ragged<DT, OT>(T, v0, tid, s);
      return;
    }
    load_chunk<true>(T, v0, tid, raw);
  }
  scale_raw<DT, OT>(T, v0, tid, s, raw);
}

template <int DT>
__device__ __forceinline__ void scale_chunk_to(const GradTensor& T, long long v0, int tid, float s,
                                               bool loaded, Raw& raw) {
  if (T.out_dtype == MUON_F32) scale_chunk<DT, MUON_F32>(T, v0, tid, s, loaded, raw);
  else if (T.out_dtype == MUON_BF16) scale_chunk<DT, MUON_BF16>(T, v0, tid, s, loaded, raw);
  else scale_chunk<DT, MUON_F16>(T, v0, tid, s, loaded, raw);
}

__device__ __forceinline__ void scale_chunk_of(const GradTensor& T, long long v0, int tid, float s,
                                               bool loaded, Raw& raw) {
  if (s == 1.f && T.out == T.g) return;   // in place and under the bound: 1 * g is g
  if (T.dtype == MUON_F32) scale_chunk_to<MUON_F32>(T, v0, tid, s, loaded, raw);
  else if (T.dtype == MUON_BF16) scale_chunk_to<MUON_BF16>(T, v0, tid, s, loaded, raw);
  else scale_chunk_to<MUON_F16>(T, v0, tid, s, loaded, raw);
}

// Chunks are taken from the last to the first: the norm read them in
// ascending order, so the last ones are the ones still in L2.  The CTA's first
// chunk is loaded before the norm is there.
template <int N>
__global__ void __launch_bounds__(GRAD_THREADS) grad_scale_kernel(const __grid_constant__ GradLaunch<N> L) {
  __shared__ unsigned long long red[GRAD_THREADS / 32];
  int c = L.nchunks - 1 - blockIdx.x;
  int ti = tensor_of(L.chunk0, L.n, c, 0);
  long long v0 = (long long)(c - L.chunk0[ti]) * GRAD_CHUNK_VECS;
  Raw raw;
  bool loaded = L.t[ti].out_vec && whole_chunk(L.t[ti], v0);
  if (loaded) load_chunk<true>(L.t[ti], v0, threadIdx.x, raw);
  pdl_wait();
  const double norm = joined(L.h, red);
  const float s = scale_of(norm, L.h);
  if (blockIdx.x == 0 && threadIdx.x == 0 && L.h.norm) write_results(L.h, norm, s);
  if (s == 1.f && L.in_place) return;
  for (;;) {
    scale_chunk_of(L.t[ti], v0, threadIdx.x, s, loaded, raw);
    c -= gridDim.x;
    if (c < 0) break;
    if (c < L.chunk0[ti]) ti = tensor_of(L.chunk0, ti, c, 0);
    v0 = (long long)(c - L.chunk0[ti]) * GRAD_CHUNK_VECS;
    loaded = false;
  }
}

// ---------------------------------------------------------------- short lists: one cluster
// Each CTA is CLUSTER_GROUPS groups of GRAD_THREADS threads; a group takes
// every (groups of the cluster)-th chunk, and reads it again to scale it (from
// L1 or L2: kept in registers it came out no faster).
constexpr int CLUSTER_GROUPS = GRAD_CLUSTER_THREADS / GRAD_THREADS;

template <int P>
__global__ void __launch_bounds__(GRAD_CLUSTER_THREADS, 1)
    grad_cluster_kernel(const __grid_constant__ GradLaunch<GRAD_SHORT_TENSORS> L) {
  __shared__ unsigned long long red[GRAD_CLUSTER_THREADS / 32];
  __shared__ unsigned long long all[GRAD_CLUSTER_MAX];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this CTA has started
  const int tid = threadIdx.x % GRAD_THREADS;
  const int group = rank * CLUSTER_GROUPS + threadIdx.x / GRAD_THREADS, groups = ctas * CLUSTER_GROUPS;
  const Acc<P> acc = block_join<P, GRAD_CLUSTER_THREADS>(add_chunks<P>(L, group, groups, tid), red);
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");             // every CTA has
  if (threadIdx.x < ctas) *cluster.map_shared_rank(&all[rank], threadIdx.x) = acc.word();
  cluster.sync();   // every CTA's value is in every CTA's `all`
  Acc<P> sum;
  for (int r = 0; r < ctas; ++r) {
    Acc<P> x;
    x.set(all[r]);
    sum.join(x);
  }
  const double norm = sum.norm();
  const float s = scale_of(norm, L.h);
  if (rank == 0 && threadIdx.x == 0) write_results(L.h, norm, s);
  if (!L.scales || (s == 1.f && L.in_place)) return;
  int ti = 0;
  for (int c = group; c < L.nchunks; c += groups) {
    ti = tensor_of(L.chunk0, L.n, c, ti);
    Raw raw;
    scale_chunk_of(L.t[ti], (long long)(c - L.chunk0[ti]) * GRAD_CHUNK_VECS, tid, s, false, raw);
  }
}

template <class F, class... A>
cudaError_t launch_with(F kernel, int grid, int threads, cudaStream_t stream, bool dependent, int cluster,
                        const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  if (dependent) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)cluster, 1, 1};
  }
  cfg.attrs = attr;
  cfg.numAttrs = dependent || cluster > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int N>
cudaError_t launch_partial(const GradLaunch<N>& L, int grid, cudaStream_t s) {
  if (L.h.norm_kind == GRAD_L1) return launch_with(grad_partial_kernel<GRAD_L1, N>, grid, GRAD_THREADS, s, false, 0, L);
  if (L.h.norm_kind == GRAD_L2) return launch_with(grad_partial_kernel<GRAD_L2, N>, grid, GRAD_THREADS, s, false, 0, L);
  return launch_with(grad_partial_kernel<GRAD_INF, N>, grid, GRAD_THREADS, s, false, 0, L);
}

}  // namespace

int grad_blocks_per_sm(bool scale) {
  int n = 0;
  const cudaError_t e =
      scale ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, grad_scale_kernel<GRAD_MAX_TENSORS>, GRAD_THREADS, 0)
            : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, grad_partial_kernel<GRAD_L2, GRAD_MAX_TENSORS>,
                                                            GRAD_THREADS, 0);
  return e != cudaSuccess || n < 1 ? 1 : n;
}

cudaError_t launch_grad_partial(const GradLaunch<GRAD_SHORT_TENSORS>& L, int grid, cudaStream_t stream) {
  return launch_partial(L, grid, stream);
}
cudaError_t launch_grad_partial(const GradLaunch<GRAD_MIDDLE_TENSORS>& L, int grid, cudaStream_t stream) {
  return launch_partial(L, grid, stream);
}
cudaError_t launch_grad_partial(const GradLaunch<GRAD_MAX_TENSORS>& L, int grid, cudaStream_t stream) {
  return launch_partial(L, grid, stream);
}
cudaError_t launch_grad_scale(const GradLaunch<GRAD_SHORT_TENSORS>& L, int grid, cudaStream_t stream) {
  return launch_with(grad_scale_kernel<GRAD_SHORT_TENSORS>, grid, GRAD_THREADS, stream, true, 0, L);
}
cudaError_t launch_grad_scale(const GradLaunch<GRAD_MIDDLE_TENSORS>& L, int grid, cudaStream_t stream) {
  return launch_with(grad_scale_kernel<GRAD_MIDDLE_TENSORS>, grid, GRAD_THREADS, stream, true, 0, L);
}
cudaError_t launch_grad_scale(const GradLaunch<GRAD_MAX_TENSORS>& L, int grid, cudaStream_t stream) {
  return launch_with(grad_scale_kernel<GRAD_MAX_TENSORS>, grid, GRAD_THREADS, stream, true, 0, L);
}
cudaError_t launch_grad_finish(const GradCall& h, cudaStream_t stream) {
  return launch_with(grad_finish_kernel, 1, GRAD_THREADS, stream, true, 0, h);
}
cudaError_t launch_grad_cluster(const GradLaunch<GRAD_SHORT_TENSORS>& L, int ctas, cudaStream_t stream) {
  if (L.h.norm_kind == GRAD_L1)
    return launch_with(grad_cluster_kernel<GRAD_L1>, ctas, GRAD_CLUSTER_THREADS, stream, false, ctas, L);
  if (L.h.norm_kind == GRAD_L2)
    return launch_with(grad_cluster_kernel<GRAD_L2>, ctas, GRAD_CLUSTER_THREADS, stream, false, ctas, L);
  return launch_with(grad_cluster_kernel<GRAD_INF>, ctas, GRAD_CLUSTER_THREADS, stream, false, ctas, L);
}

}  // namespace muon

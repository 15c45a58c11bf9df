// adamw.cu -- one AdamW step over a list of fp32 tensors in a single launch.
//
// The GPT-2 parameters that the Muon step leaves out (embeddings, LayerNorm
// gains and biases, linear biases) take AdamW.  "07. Training neural
// networks", section "Adam, weight decay and AdamW", defines the step: two
// running averages per entry (of the gradient and of its square), bias
// correction by 1 - beta^t, the move lr * u_hat / (sqrt(v_hat) + eps), and
// decoupled decay that first multiplies the parameter by (1 - lr * lambda).
//
// The work is a stream: 16 bytes read and 12 bytes written per element, no
// reuse.  So the kernel is shaped for HBM bandwidth only: persistent CTAs
// (occupancy x SM count), chunks of 2048 elements handed out in grid-stride
// order across every tensor of the call, 16-byte vector loads issued for all
// four arrays before any arithmetic so that each thread keeps eight loads in
// flight, and cache-streaming hints since nothing is read twice.  The vectors
// are the aligned ones that cover a tensor, so that one which starts off a
// 16-byte boundary takes them too, if its four arrays are off by the same (as
// views at one offset into flat buffers are); others take a scalar path with
// the same arithmetic.  39.5e6 elements in 100 tensors: 186-191 us (boxes differ),
// 5.8-5.95 TB/s, with and without a gradient scale; 30e6 elements one element off a boundary: 142
// us, as on it (208 us on the scalar path).
#include "internal.h"

namespace muon {
namespace {

// One element, in the order the page gives the step.  fp32 throughout;
// sqrtf and the division are IEEE round-to-nearest (no fast-math).
__device__ __forceinline__ void adamw_elem(float& p, float g, float& m, float& v,
                                           const AdamWLaunch& L, float decay) {
  m = fmaf(L.beta1, m, L.one_minus_beta1 * g);
  v = fmaf(L.beta2, v, L.one_minus_beta2 * (g * g));
  const float den = fmaf(sqrtf(v), L.inv_sqrt_bc2, L.eps);   // sqrt(v_hat) + eps
  p = fmaf(p, decay, -(L.step_size * m) / den);              // decay, then the Adam move
}

// The gradient the step takes: as stored, or (SCALED) times the scale, rounded
// once to fp32, so that a scaled step gives exactly what scaling the gradients
// in memory first would give.
template <bool SCALED>
__device__ __forceinline__ float taken(float g, float s) {
  return SCALED ? __fmul_rn(s, g) : g;
}

template <bool SCALED>
__device__ __forceinline__ void scalar_elem(float* P, const float* G, float* M, float* V,
                                            const AdamWLaunch& L, float decay, float s) {
  float p = __ldcs(P), g = __ldcs(G), m = __ldcs(M), v = __ldcs(V);
  adamw_elem(p, taken<SCALED>(g, s), m, v, L, decay);
  __stcs(P, p);
  __stcs(M, m);
  __stcs(V, v);
}

// Vector q of a chunk, already loaded.
template <bool SCALED>
__device__ __forceinline__ void vector_elems(int q, float* P, float* M, float* V, float4& p, const float4& g,
                                             float4& m, float4& v, const AdamWLaunch& L, float decay,
                                             float s) {
  adamw_elem(p.x, taken<SCALED>(g.x, s), m.x, v.x, L, decay);
  adamw_elem(p.y, taken<SCALED>(g.y, s), m.y, v.y, L, decay);
  adamw_elem(p.z, taken<SCALED>(g.z, s), m.z, v.z, L, decay);
  adamw_elem(p.w, taken<SCALED>(g.w, s), m.w, v.w, L, decay);
  __stcs(reinterpret_cast<float4*>(P) + q, p);
  __stcs(reinterpret_cast<float4*>(M) + q, m);
  __stcs(reinterpret_cast<float4*>(V) + q, v);
}

template <bool SCALED>
__global__ void __launch_bounds__(ADAMW_THREADS, 4) adamw_kernel(const __grid_constant__ AdamWLaunch L) {
  const float s = SCALED ? __ldg(L.grad_scale) : 1.f;
  int ti = 0;
  for (int c = blockIdx.x; c < L.nchunks; c += gridDim.x) {
    ti = tensor_of(L.chunk0, L.n, c, ti);   // chunks only grow
    const AdamWTensor& T = L.t[ti];
    // Elements are counted from the chunk's first vector; the tensor's are
    // [lo, hi) of its 2048 (lo > 0 in a first chunk that starts off a boundary).
    const long long e0 = (long long)(c - L.chunk0[ti]) * ADAMW_CHUNK - T.mis;
    const int lo = e0 < 0 ? T.mis : 0;
    const int hi = (int)min((long long)ADAMW_CHUNK, T.numel - e0);
    float* const P = T.p + e0;
    const float* const G = T.g + e0;
    float* const M = T.m + e0;
    float* const V = T.v + e0;
    if (T.vec) {
      const int q1 = hi >> 2;             // whole float4s of the chunk
      const float4* p4 = reinterpret_cast<const float4*>(P);
      const float4* g4 = reinterpret_cast<const float4*>(G);
      const float4* m4 = reinterpret_cast<const float4*>(M);
      const float4* v4 = reinterpret_cast<const float4*>(V);
      float4 p[ADAMW_VEC], g[ADAMW_VEC], m[ADAMW_VEC], v[ADAMW_VEC];
#pragma unroll
      for (int j = 0; j < ADAMW_VEC; ++j) {
        const int q = threadIdx.x + j * ADAMW_THREADS;
        if (4 * q >= lo && q < q1) {
          p[j] = __ldcs(p4 + q);
          g[j] = __ldcs(g4 + q);
          m[j] = __ldcs(m4 + q);
          v[j] = __ldcs(v4 + q);
        }
      }
#pragma unroll
      for (int j = 0; j < ADAMW_VEC; ++j) {
        const int q = threadIdx.x + j * ADAMW_THREADS;
        if (4 * q >= lo && q < q1)
          vector_elems<SCALED>(q, P, M, V, p[j], g[j], m[j], v[j], L, T.decay, s);
      }
      // The part of a last vector (threads 0..3) and of a first one (4..7),
      // once where they are the same.
      const int last = hi & ~3;
      const int e = threadIdx.x < 4 ? last + (int)threadIdx.x : (int)threadIdx.x - 4;
      const int end = threadIdx.x < 4 ? hi : (lo > 0 && last > 0 ? 4 : 0);
      if (e >= lo && e < end) scalar_elem<SCALED>(P + e, G + e, M + e, V + e, L, T.decay, s);
    } else {
      for (int e = threadIdx.x; e < hi; e += ADAMW_THREADS)
        scalar_elem<SCALED>(P + e, G + e, M + e, V + e, L, T.decay, s);
    }
  }
}

}  // namespace

int adamw_blocks_per_sm() {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, adamw_kernel<false>, ADAMW_THREADS, 0) != cudaSuccess ||
      n < 1)
    return 1;
  return n;
}

cudaError_t launch_adamw(const AdamWLaunch& L, int grid, cudaStream_t stream) {
  if (L.nchunks <= 0 || L.n <= 0) return cudaSuccess;
  if (L.grad_scale) adamw_kernel<true><<<grid, ADAMW_THREADS, 0, stream>>>(L);
  else adamw_kernel<false><<<grid, ADAMW_THREADS, 0, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace muon

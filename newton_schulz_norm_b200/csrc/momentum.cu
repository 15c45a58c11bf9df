// momentum.cu -- the HBM-bound first kernel of the Muon step, and the
// elementwise update used when no Newton-Schulz iteration runs.
//
// Per matrix (stored r x c, fp32):
//   buf <- beta*buf + g                 ("07. Training neural networks",
//                                        section "Momentum": PyTorch form)
//   u    = g + beta*buf  (Nesterov)     (X thread, tweet 5/8: orthogonalise
//   u    = buf           (plain)         the update after Nesterov momentum)
//   nu   = ||u||_F
//   X0   = bf16(u / (nu + 1e-7)), stored transposed when r > c.
//
// The norm needs the whole matrix before any element can be cast, so the
// kernel works in two passes over 64 x 64 tiles, fed by one work queue of
// items (four tiles each):
//   pass 1 (item): momentum, write buf, partial sum of squares;
//   pass 2 (item): wait until the matrix's norm is published, recompute u
//                  from g and the new buf, scale, cast, (transpose,) store.
// The host queues a matrix's pass-2 items about half a wave of CTAs after its
// last pass-1 item, behind pass-1 items of later matrices: late enough that
// the norm is usually published when they are reached, early enough that
// pass 2 re-reads g and buf mostly from L2.  The last pass-1 item of a
// matrix sums the partials in a fixed order (deterministic norm) and
// publishes it with a release store.  Pass-2 items are queued after every
// pass-1 item of their matrix, so a waiting CTA only ever waits on CTAs that
// have claimed work ahead of it; the wait is still bounded and reports
// MUON_ERR_TIMEOUT instead of hanging.
//
// A gradient scale (clipping) is one multiplication on the way in, in both
// passes; 243-246 us with it, 240-245 without on the 48 matrices of GPT-2 124M, of
// which the 14 bytes an element cannot do without take 182 us at the copy
// rate.  What u is made of (plain, momentum, Nesterov) and whether a tile is
// whole are template arguments: with both decided per element the same
// launch took 260 us, and the four matrices of one block 37.6 instead of
// 31.7 us.  Edge tiles of aligned rows load the same vectors as whole tiles, left
// out where they lie outside (200000 x 60: 55.6 us, as 200000 x 64, against 76 us
// by single elements).  Rows that are not aligned load two rows of four elements,
// neighbours in neighbouring threads, before they use the first: three matrices
// with odd sides (129 x 1001, 1003 x 129, 130 x 130) 16 instead of 49 us.  (Events
// around each launch; in a captured graph those three take 12.4 us a call, one
// 256 x 256 matrix 10.3 us.)
#include "internal.h"
#include "ptx.cuh"

namespace muon {

namespace {

// L2 residency hints.  Pass 1 loads g and buf and stores buf with an
// evict-last policy: pass 2 of the same matrix reads them again a few
// hundred work items later, and the hint keeps more of them in L2 until
// then.  Pass 2 reads them for the last time, and writes X0 (which the next
// kernel reads only after every matrix is done), with an evict-first policy.
// (Measured: about 5% faster than without hints; outputs are unchanged.)
__device__ __forceinline__ uint64_t policy_evict_last() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ float4 ld_hint(const float* a, uint64_t pol) {
  float4 v;
  asm volatile("ld.global.L2::cache_hint.v4.f32 {%0, %1, %2, %3}, [%4], %5;"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(a), "l"(pol));
  return v;
}
__device__ __forceinline__ void st_hint(float* a, float4 v, uint64_t pol) {
  asm volatile("st.global.L2::cache_hint.v4.f32 [%0], {%1, %2, %3, %4}, %5;"
               :: "l"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "l"(pol) : "memory");
}

__device__ __forceinline__ void st_hint_u2(void* a, uint2 v, uint64_t pol) {
  asm volatile("st.global.L2::cache_hint.v2.b32 [%0], {%1, %2}, %3;"
               :: "l"(a), "r"(v.x), "r"(v.y), "l"(pol) : "memory");
}
__device__ __forceinline__ void st_hint_u4(void* a, uint4 v, uint64_t pol) {
  asm volatile("st.global.L2::cache_hint.v4.b32 [%0], {%1, %2, %3, %4}, %5;"
               :: "l"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "l"(pol) : "memory");
}

__device__ __forceinline__ double block_sum(double v, double* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // red may still be read by the previous call
  if (lane == 0) red[warp] = v;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0) {
    for (int w = 0; w < K1_THREADS / 32; ++w) t += red[w];   // fixed order
  }
  return t;  // valid in thread 0 only
}

// The gradient the step takes: as stored, or (SCALED) times the launch's
// device-side scale, rounded once to fp32.  Both passes form it the same way,
// so the second one recomputes u exactly.
template <bool SCALED>
__device__ __forceinline__ float taken(float g, float s) {
  return SCALED ? __fmul_rn(s, g) : g;
}

// What u is made of.
enum Rule : int { RULE_PLAIN, RULE_MOMENTUM, RULE_NESTEROV };

template <int RULE>
__device__ __forceinline__ float momentum_u(float g, float& b, float beta) {
  if (RULE == RULE_PLAIN) return g;
  b = fmaf(beta, b, g);
  return RULE == RULE_NESTEROV ? fmaf(beta, b, g) : b;
}

template <int RULE>
__device__ __forceinline__ float u_from(float g, float bnew, float beta) {
  if (RULE == RULE_PLAIN) return g;
  return RULE == RULE_NESTEROV ? fmaf(beta, bnew, g) : bnew;
}

// How a tile is loaded.  WHOLE: it lies inside the matrix and rows are 16-byte
// aligned (c a multiple of 4), so that every group of four columns is one
// vector.  ALIGNED: the same vectors, those outside the matrix left out (a group
// is inside or outside as a whole).  LOOSE: rows are not aligned and elements
// are loaded one by one.
enum Tile : int { TILE_WHOLE, TILE_ALIGNED, TILE_LOOSE };

// The thread's four columns of rows lrow + 16 k of a tile: in vectors lcol ..
// lcol + 3, one by one every 16th, so that neighbouring threads load
// neighbouring elements.  Column e is col + e * step.
struct Cols {
  int col, step;
};

template <int TILE>
__device__ __forceinline__ Cols tile_cols(int tid) {
  const int k = tid & 15;
  return TILE == TILE_LOOSE ? Cols{k, 16} : Cols{4 * k, 1};
}

// The thread's entries of one 64 x 64 tile, RUNS rows at a time, all loaded
// before any is used; those outside the matrix are zero.  Four rows of single
// elements would cost the other tiles registers.
template <int TILE>
constexpr int RUNS = TILE == TILE_LOOSE ? 2 : 4;

struct Runs {
  float4 g[4], b[4];
};

template <int RULE, int TILE>
__device__ __forceinline__ void load_runs(const K1Ptrs& P, long long r, long long c, long long gr0,
                                          long long gc, int step, uint64_t pol, Runs& R) {
#pragma unroll
  for (int k = 0; k < RUNS<TILE>; ++k) {
    const long long gr = gr0 + 16 * k;
    const long long off = gr * c + gc;
    R.g[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    R.b[k] = R.g[k];
    if (TILE != TILE_LOOSE) {
      if (TILE == TILE_WHOLE || (gr < r && gc < c)) {
        R.g[k] = ld_hint(P.g + off, pol);
        if (RULE != RULE_PLAIN) R.b[k] = ld_hint(P.buf + off, pol);
      }
    } else {
      const bool row = gr < r, has_buf = RULE != RULE_PLAIN;
      if (row && gc < c) R.g[k].x = P.g[off];
      if (row && gc + step < c) R.g[k].y = P.g[off + step];
      if (row && gc + 2 * step < c) R.g[k].z = P.g[off + 2 * step];
      if (row && gc + 3 * step < c) R.g[k].w = P.g[off + 3 * step];
      if (row && has_buf && gc < c) R.b[k].x = __ldcg(P.buf + off);
      if (row && has_buf && gc + step < c) R.b[k].y = __ldcg(P.buf + off + step);
      if (row && has_buf && gc + 2 * step < c) R.b[k].z = __ldcg(P.buf + off + 2 * step);
      if (row && has_buf && gc + 3 * step < c) R.b[k].w = __ldcg(P.buf + off + 3 * step);
    }
  }
}

__device__ __forceinline__ int tile_kind(const K1Info& q, long long r0, long long c0) {
  if ((q.c & 3) != 0) return TILE_LOOSE;
  return r0 + K1_TILE <= q.r && c0 + K1_TILE <= q.c ? TILE_WHOLE : TILE_ALIGNED;
}

// Pass 1 on one 64 x 64 tile: momentum (buf written back) and this thread's
// sum of squares of u.  A vector of four columns sums its squares in fp32
// first; where that leaves fp32 (|u| above 9e18), they
// are formed and added in fp64, as single elements' are.  (What underflows is
// below 1e-19 an element, nothing beside the 1e-7 that the norm is added to.)
template <int RULE, bool SCALED, int TILE>
__device__ __forceinline__ double pass1_tile(const K1Launch& L, const K1Ptrs& P, long long r,
                                             long long c, long long r0, long long c0, int tid,
                                             float s, uint64_t pol) {
  const Cols C = tile_cols<TILE>(tid);
  const int lrow = tid >> 4;
  const long long gc = c0 + C.col;
  double ss = 0.0;
#pragma unroll 1
  for (int k0 = 0; k0 < 4; k0 += RUNS<TILE>) {
    Runs R;
    load_runs<RULE, TILE>(P, r, c, r0 + lrow + 16 * k0, gc, C.step, pol, R);
#pragma unroll
    for (int k = 0; k < RUNS<TILE>; ++k) {
      const long long gr = r0 + lrow + 16 * (k0 + k);
      const float gv[4] = {R.g[k].x, R.g[k].y, R.g[k].z, R.g[k].w};
      float bv[4] = {R.b[k].x, R.b[k].y, R.b[k].z, R.b[k].w};
      float u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = momentum_u<RULE>(taken<SCALED>(gv[e], s), bv[e], L.beta);
      if (TILE == TILE_WHOLE || (TILE == TILE_ALIGNED && gr < r && gc < c)) {
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) sq = fmaf(u[e], u[e], sq);
        double run = (double)sq;
        if (isinf(sq)) {
          run = 0.0;
#pragma unroll
          for (int e = 0; e < 4; ++e) run = fma((double)u[e], (double)u[e], run);
        }
        ss += run;
        if (RULE != RULE_PLAIN)
          st_hint(P.buf + gr * c + gc, make_float4(bv[0], bv[1], bv[2], bv[3]), pol);
      } else if (TILE == TILE_LOOSE && gr < r) {
        const long long off = gr * c + gc;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (gc + e * C.step < c) {
            ss += (double)u[e] * (double)u[e];
            if (RULE != RULE_PLAIN) P.buf[off + e * C.step] = bv[e];
          }
        }
      }
    }
  }
  return ss;
}

// Pass 2 on one 64 x 64 tile: recompute u from g and the new buf, scale by
// 1/(norm + eps) in double, round once to bf16 and store oriented.
template <int RULE, bool SCALED, int TILE>
__device__ __forceinline__ void pass2_tile(const K1Launch& L, const K1Ptrs& P, const K1Info& info,
                                           long long r0, long long c0, double inv, int tid,
                                           uint16_t (*s_tile)[K1_TILE + 2], float s, uint64_t pol) {
  const long long r = info.r, c = info.c;
  const bool tr = info.transposed != 0;
  const Cols C = tile_cols<TILE>(tid);
  const int lrow = tid >> 4;
#pragma unroll 1
  for (int k0 = 0; k0 < 4; k0 += RUNS<TILE>) {
    Runs R;
    load_runs<RULE, TILE>(P, r, c, r0 + lrow + 16 * k0, c0 + C.col, C.step, pol, R);
#pragma unroll
    for (int k = 0; k < RUNS<TILE>; ++k) {
      const int row = lrow + 16 * (k0 + k);
      const float gv[4] = {R.g[k].x, R.g[k].y, R.g[k].z, R.g[k].w};
      const float bv[4] = {R.b[k].x, R.b[k].y, R.b[k].z, R.b[k].w};
      uint16_t bits[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = u_from<RULE>(taken<SCALED>(gv[e], s), bv[e], L.beta);
        bits[e] = __bfloat16_as_ushort(__double2bfloat16((double)u * inv));
      }
      if (TILE != TILE_LOOSE && !tr) {
        uint2 w;
        w.x = (uint32_t)bits[0] | ((uint32_t)bits[1] << 16);
        w.y = (uint32_t)bits[2] | ((uint32_t)bits[3] << 16);
        if (TILE == TILE_WHOLE || (r0 + row < r && c0 + C.col < c))
          st_hint_u2(P.x0 + (r0 + row) * info.ldx + (c0 + C.col), w, pol);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) s_tile[row][C.col + e * C.step] = bits[e];
      }
    }
  }
  if (TILE == TILE_LOOSE && !tr) {
    // X0 row by row, four columns a thread (ldx is a multiple of 8).
    __syncthreads();
    const int col = 4 * (tid & 15);
    const long long gc = c0 + col;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = lrow + 16 * k;
      const long long gr = r0 + row;
      if (gr >= r || gc >= c) continue;
      __nv_bfloat16* dst = P.x0 + gr * info.ldx + gc;
      const uint16_t* q = &s_tile[row][col];
      if (gc + 4 <= c) {
        st_hint_u2(dst, make_uint2((uint32_t)q[0] | ((uint32_t)q[1] << 16),
                                   (uint32_t)q[2] | ((uint32_t)q[3] << 16)), pol);
      } else {
        for (int e = 0; e < 4 && gc + e < c; ++e) dst[e] = __ushort_as_bfloat16(q[e]);
      }
    }
    __syncthreads();   // s_tile is rewritten by the next tile
  }
  if (tr) {
    __syncthreads();
    // X0 row (c0 + oc) holds stored column c0 + oc; 8 threads per row.
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      const int oc = (tid >> 3) + 32 * k2;
      const int seg = (tid & 7) * 8;
      const long long xr = c0 + oc;     // row of X0 (= stored column)
      const long long xc = r0 + seg;    // first column of X0 (= stored row)
      if (xr >= c || xc >= r) continue;
      __nv_bfloat16* dst = P.x0 + xr * info.ldx + xc;
      if (xc + 8 <= r) {
        uint4 w;
        w.x = (uint32_t)s_tile[seg + 0][oc] | ((uint32_t)s_tile[seg + 1][oc] << 16);
        w.y = (uint32_t)s_tile[seg + 2][oc] | ((uint32_t)s_tile[seg + 3][oc] << 16);
        w.z = (uint32_t)s_tile[seg + 4][oc] | ((uint32_t)s_tile[seg + 5][oc] << 16);
        w.w = (uint32_t)s_tile[seg + 6][oc] | ((uint32_t)s_tile[seg + 7][oc] << 16);
        st_hint_u4(dst, w, pol);
      } else {
        for (int e = 0; e < 8 && xc + e < r; ++e) dst[e] = __ushort_as_bfloat16(s_tile[seg + e][oc]);
      }
    }
    __syncthreads();   // s_tile is rewritten by the next tile
  }
}

template <int RULE, bool SCALED>
__global__ void __launch_bounds__(K1_THREADS, 4) k1_kernel(const __grid_constant__ K1Launch L) {
  __shared__ int s_item;
  __shared__ int s_flag;
  __shared__ double s_norm;
  __shared__ double s_red[K1_THREADS / 32];
  __shared__ uint16_t s_tile[K1_TILE][K1_TILE + 2];

  const int tid = threadIdx.x;
  const float s = SCALED ? __ldg(L.grad_scale) : 1.f;
  const uint64_t pol_keep = policy_evict_last();
  const uint64_t pol_drop = policy_evict_first();

  for (;;) {
    if (tid == 0) s_item = atomicAdd(L.counter, 1);
    __syncthreads();
    const int it = s_item;
    __syncthreads();
    if (it >= L.nitems) break;
    const K1Item item = L.items[it];
    const bool pass2 = (item.mat & K1_PASS2) != 0;
    const int mat = item.mat & ~K1_PASS2;
    if (kBoundsCheck) {
      // Checked builds: the item must name a matrix of the launch and one of
      // its groups, whose partial sum lies inside the partials array.
      bool ok = mat >= 0 && mat < L.n;
      if (ok) {
        const K1Info& q = L.info[mat];
        ok = item.group >= 0 && item.group < q.nitems && q.part0 >= 0 &&
             (long long)q.part0 + q.nitems <= L.npartials;
      }
      if (!ok) {
        if (tid == 0) atomicCAS(L.status, 0, MUON_ERR_INVALID_ARG);
        continue;
      }
    }
    const K1Info info = L.info[mat];
    const K1Ptrs P = L.ptrs[mat];
    const int t0 = item.group * info.group;
    const int t1 = min(t0 + info.group, info.ntiles);

    if (!pass2) {
      double ss = 0.0;
      for (int t = t0; t < t1; ++t) {
        const long long r0 = (long long)(t / info.tiles_c) * K1_TILE;
        const long long c0 = (long long)(t % info.tiles_c) * K1_TILE;
        const int kind = tile_kind(info, r0, c0);
        if (kind == TILE_WHOLE)
          ss += pass1_tile<RULE, SCALED, TILE_WHOLE>(L, P, info.r, info.c, r0, c0, tid, s, pol_keep);
        else if (kind == TILE_ALIGNED)
          ss += pass1_tile<RULE, SCALED, TILE_ALIGNED>(L, P, info.r, info.c, r0, c0, tid, s, pol_keep);
        else
          ss += pass1_tile<RULE, SCALED, TILE_LOOSE>(L, P, info.r, info.c, r0, c0, tid, s, pol_keep);
      }
      const double tot = block_sum(ss, s_red);
      if (tid == 0) {
        L.partials[info.part0 + item.group] = tot;
        // Release: this CTA's buf stores (ordered before by the barriers in
        // block_sum) and the partial become visible before the count does.
        __threadfence();
        const int prev = atomicAdd(L.done + mat, 1);
        s_flag = (prev == info.nitems - 1);
      }
      __syncthreads();
      if (s_flag) {
        // Last item of this matrix: fixed-order sum of its partials.
        __threadfence();
        double acc = 0.0;
        for (int t = tid; t < info.nitems; t += K1_THREADS) acc += __ldcg(L.partials + info.part0 + t);
        const double all = block_sum(acc, s_red);
        if (tid == 0) {
          L.norms[mat] = sqrt(all);
          __threadfence();
          st_release_gpu(L.ready + mat, 1);
        }
      }
      continue;
    }

    // ---------------------------------------------------------------- pass 2
    if (tid == 0) {
      int ok = ld_acquire_gpu(L.ready + mat);
      if (!ok) {
        const uint64_t t0ns = global_timer_ns();
        while (!(ok = ld_acquire_gpu(L.ready + mat))) {
          if (global_timer_ns() - t0ns > L.limit_ns) break;
          __nanosleep(128);
        }
      }
      if (!ok) atomicCAS(L.status, 0, MUON_ERR_TIMEOUT);
      s_flag = ok;
      s_norm = ok ? __ldcg(L.norms + mat) : 0.0;
    }
    __syncthreads();
    if (!s_flag) continue;
    const double inv = 1.0 / (s_norm + 1e-7);
    for (int t = t0; t < t1; ++t) {
      const long long r0 = (long long)(t / info.tiles_c) * K1_TILE;
      const long long c0 = (long long)(t % info.tiles_c) * K1_TILE;
      const int kind = tile_kind(info, r0, c0);
      if (kind == TILE_WHOLE)
        pass2_tile<RULE, SCALED, TILE_WHOLE>(L, P, info, r0, c0, inv, tid, s_tile, s, pol_drop);
      else if (kind == TILE_ALIGNED)
        pass2_tile<RULE, SCALED, TILE_ALIGNED>(L, P, info, r0, c0, inv, tid, s_tile, s, pol_drop);
      else
        pass2_tile<RULE, SCALED, TILE_LOOSE>(L, P, info, r0, c0, inv, tid, s_tile, s, pol_drop);
    }
  }
}

// p <- p - scale * X0 (or a plain copy of X0 out) for ns_steps == 0.
__global__ void apply_kernel(const __grid_constant__ ApplyLaunch L) {
  const int mat = blockIdx.y;
  if (mat >= L.n) return;
  const K1Info info = L.info[mat];
  const long long r = info.r, c = info.c, total = r * c;
  const __nv_bfloat16* x0 = L.ptrs[mat].x0;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (long long)gridDim.x * blockDim.x) {
    const long long i = e / c, j = e % c;                 // stored position
    const long long xo = info.transposed ? (j * info.ldx + i) : (i * info.ldx + j);
    const float x = __bfloat162float(x0[xo]);
    if (L.mode == FINAL_PARAM) {
      float* p = reinterpret_cast<float*>(L.dst[mat]) + e;
      *p = __fadd_rn(*p, __fmul_rn(-L.scale[mat], x));   // p + fp32(-s x), as the GEMM paths
    } else if (L.mode == FINAL_OUT_F32) {
      reinterpret_cast<float*>(L.dst[mat])[e] = x;
    } else {
      reinterpret_cast<__nv_bfloat16*>(L.dst[mat])[e] = __float2bfloat16_rn(x);
    }
  }
}

typedef void (*K1Kernel)(const K1Launch);

K1Kernel k1_kernel_for(int mode, int nesterov, bool scaled) {
  if (mode == K1_PLAIN) return k1_kernel<RULE_PLAIN, false>;
  if (nesterov) return scaled ? k1_kernel<RULE_NESTEROV, true> : k1_kernel<RULE_NESTEROV, false>;
  return scaled ? k1_kernel<RULE_MOMENTUM, true> : k1_kernel<RULE_MOMENTUM, false>;
}

}  // namespace

int k1_blocks_per_sm() {
  int least = 0;
  for (int k = 0; k < 5; ++k) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &n, k1_kernel_for(k == 4 ? K1_PLAIN : K1_MOMENTUM, k & 1, (k & 2) != 0), K1_THREADS, 0) !=
            cudaSuccess ||
        n < 1)
      return 1;
    least = k == 0 || n < least ? n : least;
  }
  return least;
}

cudaError_t launch_k1(const K1Launch& L, int grid, cudaStream_t stream) {
  if (L.nitems <= 0) return cudaSuccess;
  k1_kernel_for(L.mode, L.nesterov, L.grad_scale != nullptr)<<<grid, K1_THREADS, 0, stream>>>(L);
  return cudaGetLastError();
}

cudaError_t launch_apply(const ApplyLaunch& L, cudaStream_t stream) {
  if (L.n <= 0) return cudaSuccess;
  apply_kernel<<<dim3(256, L.n), 256, 0, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace muon

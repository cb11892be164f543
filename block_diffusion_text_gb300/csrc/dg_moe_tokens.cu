// A layer's whole mixture-of-experts block for a few tokens, in one launch:
//
//   x = RMSNorm(h), r = x Wr^T, e_j = the top_k experts of r, g = softmax of their r
//   out = h + sum_j g_j We2_ej GELU(We1_ej x) + We2_s GELU(We1_s x)
//
// The chosen experts' weights bound it: each matrix is read once, whatever the
// number of tokens that chose it.  One persistent CTA per SM works through three
// phases with a barrier of the grid between them, as the data demands:
//   0  router logits, and the shared expert's hidden rows (they need no routing)
//   1  every CTA works the routing out for itself; the chosen experts' hidden rows
//   2  the output columns
// In each phase the rows of the weights that it needs are cut into equal ranges,
// one for each CTA, row by row, so that all SMs read the same number of bytes.
//
// Warp MMAs, the weights as the 16-row operand, the tokens as the columns; a row of
// 32 tokens is four column tiles, and those without a token of the expert are
// skipped.  x W^T is taken as (h W^T) / rms, so the tokens enter as the bf16 they
// are; the hidden values, which carry their gate (the second product is linear), as
// pairs of bf16 (16 bits or more).  A warp's share of the products' inner dimension
// is a block of 64 columns in turn; its own weights come through a ring of cp.async
// copies that only the lane that issued them reads, so nothing has to be waited for
// but the lane's own copies.
#include <cfloat>
#include <climits>

#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kMtWarps = 16;
constexpr int kMtThreads = kMtWarps * 32;
constexpr int kMtStages = 4;
constexpr int kMtStage = 2048;  // 16 rows of 64 columns
constexpr int kMtMaxM = 32;
constexpr int kMtMaxExp = 256, kMtMaxK = 16;

struct MtArgs {
  const __nv_bfloat16* h;                  // [M][d]
  __nv_bfloat16* out;                      // [M][d], may be h
  const __nv_bfloat16 *Wr, *W1, *W2;       // [n_exp][d], [n_exp + 1][Fe][d], [n_exp + 1][d][Fe]
  float* logits;                           // [M][n_exp]
  __nv_bfloat16 *hi, *lo;                  // [M][top_k + 1][Fe]: gate GELU(x We1^T)
  int* idx;                                // [M][top_k] or null
  float* gate;                             // [M][top_k] or null
  int* status;
  unsigned* bar;                           // arrivals, rounds
  int M, d, Fe, n_exp, top_k;
  float eps;
};

struct MtShared {
  float inv[kMtMaxM];
  float gate[kMtMaxM][kMtMaxK];
  unsigned mask[kMtMaxExp];                // tokens of an expert
  uint8_t rank[kMtMaxExp][kMtMaxM];        // their place among the token's experts
  int act[kMtMaxExp];                      // the experts with tokens, ascending
  int nact;
  int stop;
};

// All CTAs of the grid are here (the launch is cooperative).  Thread 0 arrives for
// its CTA; the last one to arrive begins the next round.  Bounded: false, with the
// status word set, if the others do not come.
DG_DEV bool grid_barrier(unsigned* bar, int* status, int* stop) {
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned round;
    asm volatile("ld.relaxed.gpu.u32 %0, [%1];" : "=r"(round) : "l"(bar + 1) : "memory");
    __threadfence();
    if (atomicAdd(bar, 1u) == gridDim.x - 1) {
      *reinterpret_cast<volatile unsigned*>(bar) = 0u;
      __threadfence();
      atomicAdd(bar + 1, 1u);
    } else {
      uint64_t t0 = 0;
      for (unsigned i = 0;; ++i) {
        unsigned now;
        asm volatile("ld.relaxed.gpu.u32 %0, [%1];" : "=r"(now) : "l"(bar + 1) : "memory");
        if (now != round) break;
        if (i % 256 == 255) {
          if (!t0) t0 = globaltimer();
          else if (globaltimer() - t0 > kWaitLimitNs) {
            atomicExch(status, kStatusTimeout);
            *stop = 1;
            break;
          }
        }
      }
    }
    __threadfence();
  }
  __syncthreads();
  return *stop == 0;
}

DG_DEV void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

DG_DEV float gelu(float x) { return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f)); }

// Stage of a ring: the lane's pieces of rows g and g + 8, halves 0 and 1 of the 64
// columns.  Rows at or past `rows` are not copied: what their products hold is not used.
DG_DEV void load_block(char* slot, const __nv_bfloat16* w, int64_t pitch, int rows, int lane) {
  const int g = lane / 4, t = lane % 4;
#pragma unroll
  for (int r = 0; r < 2; ++r)
    if (g + 8 * r < rows) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
        cp_async16(slot + ((r * 2 + p) * 32 + lane) * 16, w + (g + 8 * r) * pitch + 32 * p + 8 * t);
    }
}

// The products of one block: acc[n] += (16 rows) x (8 tokens), b(n, p) the lane's
// eight values of its token in half p.
template <int NT, class B>
DG_DEV void block_products(float (&acc)[NT][4], const char* slot, int lane, unsigned tiles, const B& b) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint4 u = *reinterpret_cast<const uint4*>(slot + (p * 32 + lane) * 16);
    const uint4 v = *reinterpret_cast<const uint4*>(slot + ((2 + p) * 32 + lane) * 16);
    const uint32_t A0[4] = {u.x, v.x, u.y, v.y}, A1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (tiles >> n & 1) b(acc[n], n, p, A0, A1);
  }
}

DG_DEV unsigned tiles_of(unsigned mask) {  // a bit for each eight tokens that hold one
  return (mask & 0xffu ? 1u : 0u) | (mask & 0xff00u ? 2u : 0u) | (mask & 0xff0000u ? 4u : 0u) | (mask & 0xff000000u ? 8u : 0u);
}

template <int NT>
__global__ void __launch_bounds__(kMtThreads, 1) moe_tokens_kernel(MtArgs a) {
  extern __shared__ __align__(16) char smem[];
  char* ring = smem + (threadIdx.x / 32) * kMtStages * kMtStage;
  float* red = reinterpret_cast<float*>(smem + kMtWarps * kMtStages * kMtStage);  // [warps][NT * 4][32]
  __shared__ MtShared s;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int K1 = a.top_k + 1, KB1 = a.d / 64, KB2 = a.Fe / 64;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const unsigned all = a.M == 32 ? 0xffffffffu : (1u << a.M) - 1;
  if (tid == 0) s.stop = 0;

  // 1 / rms of every token, for this CTA's own use
  for (int m = warp; m < a.M; m += kMtWarps) {
    float sum = 0.f;
    const uint4* src = reinterpret_cast<const uint4*>(a.h + (size_t)m * a.d);
    for (int i = lane; i < a.d / 8; i += 32) {
      const uint4 v = src[i];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = __uint_as_float(w[j] << 16), y = __uint_as_float(w[j] & 0xffff0000u);
        sum += x * x + y * y;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s.inv[m] = 1.0f / sqrtf(sum / (float)a.d + a.eps);
  }
  __syncthreads();

  // The sums of a unit over the CTA's warps, in order; thread i * 32 + lane gets the
  // value of (row g + 8 (i % 4 / 2), token 8 (i / 4) + 2 t + i % 2).
  auto unit_sum = [&](const float (&acc)[NT][4], const auto& put) {
#pragma unroll
    for (int i = 0; i < NT * 4; ++i) red[(warp * NT * 4 + i) * 32 + lane] = acc[i / 4][i % 4];
    __syncthreads();
    if (tid < NT * 128) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kMtWarps; ++w) v += red[w * NT * 128 + tid];
      const int i = tid / 32;
      put(g + 8 * (i % 4 / 2), 8 * (i / 4) + 2 * t + i % 2, v);
    }
    __syncthreads();
  };

  // Products of h with rows [r0, r1) of a row space cut into tiles of 16: unit u is
  // tile r0 / 16 + u.  src(tile) is the tile's first row in memory and the tokens that
  // want it; put(row of the space, token, sum).
  auto rows_of_h = [&](int r0, int r1, const auto& src, const auto& put) {
    if (r1 <= r0) return;
    const int T0 = r0 / 16, U = (r1 + 15) / 16 - T0;
    const int total = U * KB1;
    auto issue = [&](int i, int slot) {
      if (i < total) {
        const int u = i / KB1, kb = i % KB1, lo = max(r0, 16 * (T0 + u)), hi = min(r1, 16 * (T0 + u) + 16);
        const __nv_bfloat16* w;
        int rows;
        unsigned mask;
        src(T0 + u, &w, &rows, &mask);
        const int skip = lo - 16 * (T0 + u);
        rows = min(rows - skip, hi - lo);
        load_block(ring + slot * kMtStage, w + (int64_t)skip * a.d + kb * 64, a.d, rows, lane);
      }
      cp_async_commit();
    };
    int i = warp, put_slot = 0, get_slot = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < kMtStages - 1; ++s0) {
      issue(i + s0 * kMtWarps, put_slot);
      put_slot = put_slot + 1 == kMtStages ? 0 : put_slot + 1;
    }
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
      float acc[NT][4] = {};
      const __nv_bfloat16* w;
      int rows;
      unsigned mask;
      src(T0 + u, &w, &rows, &mask);
      const unsigned tiles = tiles_of(mask);
#pragma unroll 1
      for (; i < (u + 1) * KB1; i += kMtWarps) {
        issue(i + (kMtStages - 1) * kMtWarps, put_slot);
        put_slot = put_slot + 1 == kMtStages ? 0 : put_slot + 1;
        cp_async_wait<kMtStages - 1>();
        const __nv_bfloat16* x = a.h + (i - u * KB1) * 64 + 8 * t;
        block_products<NT>(acc, ring + get_slot * kMtStage, lane, tiles,
                           [&](float(&c)[4], int n, int p, const uint32_t(&A0)[4], const uint32_t(&A1)[4]) {
                             uint4 b = make_uint4(0, 0, 0, 0);
                             if (mask >> (8 * n + g) & 1)
                               b = *reinterpret_cast<const uint4*>(x + (int64_t)(8 * n + g) * a.d + 32 * p);
                             mma_bf16_16816(c, A0, b.x, b.y);
                             mma_bf16_16816(c, A1, b.z, b.w);
                           });
        get_slot = get_slot + 1 == kMtStages ? 0 : get_slot + 1;
      }
      const int lo = max(r0, 16 * (T0 + u)), hi = min(r1, 16 * (T0 + u) + 16);
      unit_sum(acc, [&](int row, int m, float v) {
        if (lo + row < hi && (mask >> m & 1)) put(lo + row, m, v * s.inv[m]);
      });
    }
    cp_async_wait<0>();
  };
  auto range = [&](int rows, int c) { return (int)((int64_t)rows * c / ctas); };
  auto store_hidden = [&](int m, int j, int f, float v) {
    const size_t at = ((size_t)m * K1 + j) * a.Fe + f;
    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
    a.hi[at] = hi;
    a.lo[at] = __float2bfloat16_rn(v - __bfloat162float(hi));
  };

  // ---- phase 0: the router's rows, then the shared expert's
  const int n16 = (a.n_exp + 15) / 16 * 16;
  rows_of_h(
      range(n16 + a.Fe, cta), range(n16 + a.Fe, cta + 1),
      [&](int tile, const __nv_bfloat16** w, int* rows, unsigned* mask) {
        const bool router = 16 * tile < n16;
        *w = router ? a.Wr + (int64_t)tile * 16 * a.d : a.W1 + ((int64_t)a.n_exp * a.Fe + 16 * tile - n16) * a.d;
        *rows = router ? min(16, a.n_exp - 16 * tile) : 16;
        *mask = all;
      },
      [&](int row, int m, float v) {
        if (row < a.n_exp) a.logits[(size_t)m * a.n_exp + row] = v;
        else if (row >= n16) store_hidden(m, a.top_k, row - n16, gelu(v));
      });
  if (!grid_barrier(a.bar, a.status, &s.stop)) return;

  // ---- the routing: one warp for each token, a lane holding experts lane, lane + 32, ..
  for (int e = tid; e < kMtMaxExp; e += kMtThreads) s.mask[e] = 0;
  __syncthreads();
  for (int m = warp; m < a.M; m += kMtWarps) {
    float l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) l[j] = lane + 32 * j < a.n_exp ? __ldcg(a.logits + (size_t)m * a.n_exp + lane + 32 * j) : 0.f;
    uint32_t taken = 0;
    float top = 0.f, Z = 0.f, mine = 0.f;
    int mye = 0;
#pragma unroll 1
    for (int k = 0; k < a.top_k; ++k) {
      float bv = -FLT_MAX;
      int be = INT_MAX;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = lane + 32 * j;
        if (e < a.n_exp && !((taken >> j) & 1u) && (l[j] > bv || (l[j] == bv && e < be))) {
          bv = l[j];
          be = e;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
        const int oe = __shfl_xor_sync(0xffffffffu, be, o);
        if (ov > bv || (ov == bv && oe < be)) {
          bv = ov;
          be = oe;
        }
      }
      if (be >= a.n_exp || !(bv <= FLT_MAX)) {  // non-finite logits: recorded
        if (lane == 0 && cta == 0) atomicExch(a.status, kStatusValue);
        if (be >= a.n_exp) {  // none is left that compares: the lowest one not taken
          bv = -FLT_MAX;
          int first = INT_MAX;
#pragma unroll
          for (int j = 7; j >= 0; --j)
            if (lane + 32 * j < a.n_exp && !((taken >> j) & 1u)) first = lane + 32 * j;
          be = (int)__reduce_min_sync(0xffffffffu, (unsigned)first);
        }
      }
      if ((be & 31) == lane) taken |= 1u << (be >> 5);
      if (k == 0) top = bv;
      Z += expf(bv - top);
      if (lane == k) {
        mine = bv;
        mye = be;
      }
    }
    if (lane < a.top_k) {
      const float gt = expf(mine - top) / Z;
      s.gate[m][lane] = gt;
      s.rank[mye][m] = (uint8_t)lane;
      atomicOr(&s.mask[mye], 1u << m);
      if (cta == 0) {
        if (a.idx) a.idx[(size_t)m * a.top_k + lane] = mye;
        if (a.gate) a.gate[(size_t)m * a.top_k + lane] = gt;
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int e0 = 0; e0 < a.n_exp; e0 += 32) {
      const bool on = e0 + lane < a.n_exp && s.mask[e0 + lane] != 0;
      const unsigned b = __ballot_sync(0xffffffffu, on);
      if (on) s.act[n + __popc(b & ((1u << lane) - 1))] = e0 + lane;
      n += __popc(b);
    }
    if (lane == 0) s.nact = n;
  }
  __syncthreads();
  const int nact = s.nact;

  // ---- phase 1: the chosen experts' hidden rows
  const int R1 = nact * a.Fe;
  rows_of_h(
      range(R1, cta), range(R1, cta + 1),
      [&](int tile, const __nv_bfloat16** w, int* rows, unsigned* mask) {
        const int e = s.act[16 * tile / a.Fe];
        *w = a.W1 + ((int64_t)e * a.Fe + 16 * tile % a.Fe) * a.d;
        *rows = 16;
        *mask = s.mask[e];
      },
      [&](int row, int m, float v) {
        const int e = s.act[row / a.Fe], j = s.rank[e][m];
        store_hidden(m, j, row % a.Fe, s.gate[m][j] * gelu(v));
      });
  if (!grid_barrier(a.bar, a.status, &s.stop)) return;

  // ---- phase 2: output columns [r0, r1), their sums over the experts' hidden values
  {
    const int r0 = range(a.d, cta), r1 = range(a.d, cta + 1);
    const int U = (r1 - r0 + 15) / 16, items = (nact + 1) * KB2;
    const int64_t total = (int64_t)U * items;
    auto issue = [&](int64_t i, int slot) {
      if (i < total) {
        const int u = (int)(i / items), at = (int)(i % items), x = at / KB2, kb = at % KB2;
        const int e = x < nact ? s.act[x] : a.n_exp, row = r0 + 16 * u;
        load_block(ring + slot * kMtStage, a.W2 + ((int64_t)e * a.d + row) * a.Fe + kb * 64, a.Fe, r1 - row, lane);
      }
      cp_async_commit();
    };
    int64_t i = warp;
    int put_slot = 0, get_slot = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < kMtStages - 1; ++s0) {
      issue(i + s0 * kMtWarps, put_slot);
      put_slot = put_slot + 1 == kMtStages ? 0 : put_slot + 1;
    }
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
      float acc[NT][4] = {};
#pragma unroll 1
      for (; i < (int64_t)(u + 1) * items; i += kMtWarps) {
        issue(i + (kMtStages - 1) * kMtWarps, put_slot);
        put_slot = put_slot + 1 == kMtStages ? 0 : put_slot + 1;
        cp_async_wait<kMtStages - 1>();
        const int at = (int)(i - (int64_t)u * items), x = at / KB2, kb = at % KB2;
        const int e = x < nact ? s.act[x] : a.n_exp;
        const unsigned mask = x < nact ? s.mask[e] : all;
        block_products<NT>(acc, ring + get_slot * kMtStage, lane, tiles_of(mask),
                           [&](float(&c)[4], int n, int p, const uint32_t(&A0)[4], const uint32_t(&A1)[4]) {
                             uint4 b = make_uint4(0, 0, 0, 0), bl = b;
                             const int m = 8 * n + g;
                             if (mask >> m & 1) {
                               const int j = x < nact ? s.rank[e][m] : a.top_k;
                               const size_t off = ((size_t)m * K1 + j) * a.Fe + kb * 64 + 32 * p + 8 * t;
                               b = *reinterpret_cast<const uint4*>(a.hi + off);
                               bl = *reinterpret_cast<const uint4*>(a.lo + off);
                             }
                             mma_bf16_16816(c, A0, b.x, b.y);
                             mma_bf16_16816(c, A1, b.z, b.w);
                             mma_bf16_16816(c, A0, bl.x, bl.y);
                             mma_bf16_16816(c, A1, bl.z, bl.w);
                           });
        get_slot = get_slot + 1 == kMtStages ? 0 : get_slot + 1;
      }
      const int row0 = r0 + 16 * u;
      unit_sum(acc, [&](int row, int m, float v) {
        if (row0 + row < r1 && m < a.M) {
          const size_t at = (size_t)m * a.d + row0 + row;
          a.out[at] = __float2bfloat16_rn(__bfloat162float(a.h[at]) + v);
        }
      });
    }
    cp_async_wait<0>();
  }
}

struct MtWs {
  size_t logits, hi, lo, total;
};

MtWs mt_ws(int M, int n_exp, int top_k, int Fe) {
  MtWs w;
  size_t o = 256;  // status word, the barrier's two words
  w.logits = o;
  o = align_up(o + sizeof(float) * M * n_exp, 256);
  w.hi = o;
  o = align_up(o + 2 * (size_t)M * (top_k + 1) * Fe, 256);
  w.lo = o;
  o = align_up(o + 2 * (size_t)M * (top_k + 1) * Fe, 256);
  w.total = o;
  return w;
}

dg_status check_sizes(const dg_model* m, int32_t M) {
  if (!m) return DG_ERR_ARG;
  const dg_dims& D = m->dims;
  if (M <= 0 || D.d <= 0 || D.n_exp <= 0 || D.top_k <= 0 || D.top_k > D.n_exp || D.Fe <= 0 || D.L <= 0 || !(D.rms_eps >= 0.f))
    return DG_ERR_ARG;
  if (M > kMtMaxM || D.d % 128 || D.d > 16384 || D.Fe % 128 || D.Fe > 16384 || D.n_exp > kMtMaxExp || D.top_k > kMtMaxK || D.L > 64)
    return DG_ERR_SHAPE;
  return DG_OK;
}

template <int NT>
cudaError_t launch(const MtArgs& a, int sms, cudaStream_t st) {
  const int smem = kMtWarps * kMtStages * kMtStage + kMtWarps * NT * 4 * 32 * (int)sizeof(float);
  cudaError_t e = set_smem_once<moe_tokens_kernel<NT>>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(kMtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_tokens_kernel<NT>, a);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" dg_status dg_moe_tokens_workspace(const dg_model* model, int32_t M, size_t* bytes) {
  if (!bytes) return DG_ERR_ARG;
  dg_status e = check_sizes(model, M);
  if (e) return e;
  *bytes = mt_ws(M, model->dims.n_exp, model->dims.top_k, model->dims.Fe).total;
  return DG_OK;
}

extern "C" dg_status dg_moe_tokens(const dg_model* model, int32_t layer, const void* h, void* out, int32_t M, int32_t* idx,
                                   float* gate, void* ws, size_t ws_bytes, void* stream) {
  dg_status s = check_sizes(model, M);
  if (s) return s;
  const dg_dims& D = model->dims;
  if (layer < 0 || layer >= D.L || !h || !out || !ws || !model->Wr || !model->We1 || !model->We2) return DG_ERR_ARG;
  if (!aligned16(h) || !aligned16(out) || !aligned16(model->Wr) || !aligned16(model->We1) || !aligned16(model->We2) ||
      reinterpret_cast<uintptr_t>(idx) % 4 || reinterpret_cast<uintptr_t>(gate) % 4)
    return DG_ERR_ARG;
  const MtWs w = mt_ws(M, D.n_exp, D.top_k, D.Fe);
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < w.total) return DG_ERR_WORKSPACE;
  uint8_t* base = static_cast<uint8_t*>(ws);
  const size_t e1 = (size_t)(D.n_exp + 1) * D.Fe * D.d;
  MtArgs a{};
  a.h = static_cast<const __nv_bfloat16*>(h);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.Wr = static_cast<const __nv_bfloat16*>(model->Wr) + layer * (size_t)D.n_exp * D.d;
  a.W1 = static_cast<const __nv_bfloat16*>(model->We1) + layer * e1;
  a.W2 = static_cast<const __nv_bfloat16*>(model->We2) + layer * e1;
  a.logits = reinterpret_cast<float*>(base + w.logits);
  a.hi = reinterpret_cast<__nv_bfloat16*>(base + w.hi);
  a.lo = reinterpret_cast<__nv_bfloat16*>(base + w.lo);
  a.idx = idx;
  a.gate = gate;
  a.status = reinterpret_cast<int*>(base);
  a.bar = reinterpret_cast<unsigned*>(base + 64);
  a.M = M;
  a.d = D.d;
  a.Fe = D.Fe;
  a.n_exp = D.n_exp;
  a.top_k = D.top_k;
  a.eps = D.rms_eps;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DG_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = M <= 8 ? launch<1>(a, sms, st) : M <= 16 ? launch<2>(a, sms, st) : launch<4>(a, sms, st);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

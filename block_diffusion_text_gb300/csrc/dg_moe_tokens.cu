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
#include <type_traits>

#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kMtWarps = 16;
constexpr int kMtThreads = kMtWarps * 32;
constexpr int kMtStages = 2;
constexpr int kMtRows = 32;     // rows of a unit: two MMA tiles
constexpr int kMtStage = kMtRows * 128;  // 64 columns of them
constexpr int kMtRed = 65536;   // shared memory for the warps' parts of units' sums
constexpr int kMtMaxM = 32;
constexpr int kMtMaxExp = 256, kMtMaxK = 16;

struct MtArgs {
  const __nv_bfloat16* h;                  // [M][d]
  __nv_bfloat16* out;                      // [M][d], may be h
  const __nv_bfloat16 *Wr, *W1, *W2;       // [n_exp][d], [n_exp + 1][Fe][d], [n_exp + 1][d][Fe]
  float* logits;                           // [M][n_exp]
  __nv_bfloat16* hid;                      // [M (top_k + 1) + 1][Fe / 32][2][32]: gate GELU(x We1^T), the values as
                                           // bf16 and what that leaves; the last row is zeros
  int* idx;                                // [M][top_k] or null
  float* gate;                             // [M][top_k] or null
  int* status;
  unsigned* bar;                           // arrivals, rounds
  int M, d, Fe, n_exp, top_k;
  float eps;
};

struct MtExpert {
  int e;
  unsigned mask;                           // its tokens
};

struct MtShared {
  float inv[kMtMaxM];
  float gate[kMtMaxM][kMtMaxK];
  unsigned mask[kMtMaxExp];                // tokens of every expert
  uint8_t place[kMtMaxExp][kMtMaxM];       // their place among the token's experts
  MtExpert ex[kMtMaxExp + 1];              // the experts with tokens, ascending, and the shared one
  uint8_t rank[kMtMaxExp + 1][kMtMaxM];    // and the place of each of their tokens
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

// Stage of a ring: the lane's pieces of rows g, g + 8, g + 16 and g + 24, halves 0 and
// 1 of the 64 columns.  Rows at or past `rows` are not copied: what their products
// hold is not used.
DG_DEV void load_block(char* slot, const __nv_bfloat16* w, int pitch, int rows, int lane) {
  const int g = lane / 4, t = lane % 4;
  const __nv_bfloat16* src = w + g * pitch + 8 * t;
#pragma unroll
  for (int r = 0; r < kMtRows / 8; ++r)
    if (g + 8 * r < rows) {
#pragma unroll
      for (int p = 0; p < 2; ++p) cp_async16(slot + ((r * 2 + p) * 32 + lane) * 16, src + 8 * r * pitch + 32 * p);
    }
}

DG_DEV unsigned tiles_of(unsigned mask) {  // a bit for each eight tokens that hold one
  return (mask & 0xffu ? 1u : 0u) | (mask & 0xff00u ? 2u : 0u) | (mask & 0xff0000u ? 4u : 0u) | (mask & 0xff000000u ? 8u : 0u);
}

// Rows [r0, r1) cut into units of 32 rows at most, from r0 to the border rb (a
// matrix's end) and from there on.  (Further matrices begin at multiples of 32 from
// there: their rows are multiples of 128.)
struct MtCut {
  int r0, rb, r1, U0, U;
  DG_DEV MtCut() {}
  DG_DEV MtCut(int first, int end, int border) : r0(first), r1(end) {
    rb = border > first && border < end ? border : end;
    U0 = (rb - r0 + kMtRows - 1) / kMtRows;
    U = U0 + (r1 - rb + kMtRows - 1) / kMtRows;
  }
  DG_DEV int row(int u) const { return u < U0 ? r0 + kMtRows * u : rb + kMtRows * (u - U0); }
  DG_DEV int rows(int u) const { return min(kMtRows, (u < U0 ? rb : r1) - row(u)); }
};

// Cursors over the segments of a CTA's units: of the router and the shared expert,
// of the chosen experts (both multiply the tokens themselves), and of the second
// matrices.
template <int NT>
struct RowsOfH0 {
  MtCut cut;
  const __nv_bfloat16 *Wr, *Ws, *w;
  int border, n_exp, d, u, rows;
  unsigned tiles;
  int off[NT];
  DG_DEV void start(int g, int t, int M) {
    tiles = (1u << ((M + 7) / 8)) - 1;
#pragma unroll
    for (int n = 0; n < NT; ++n) off[n] = min(8 * n + g, M - 1) * d + 8 * t;  // columns past the last token repeat it
    u = -1;
    next();
  }
  DG_DEV void next() {
    if (++u >= cut.U) return;
    const int r = cut.row(u);
    rows = r < border ? min(cut.rows(u), n_exp - r) : cut.rows(u);
    w = r < border ? Wr + (int64_t)r * d : Ws + (int64_t)(r - border) * d;
  }
};

// A column whose token does not want the expert takes the values of one that does:
// its sum is not stored.
template <int NT>
struct RowsOfH1 {
  MtCut cut;
  const __nv_bfloat16 *W1, *w;
  const MtExpert* ex;
  int F, d, u, rows, g, t;
  unsigned tiles;
  int off[NT];
  DG_DEV void start() {
    u = -1;
    next();
  }
  DG_DEV void next() {
    if (++u >= cut.U) return;
    const int r = cut.row(u), x = r / F;
    const MtExpert e = ex[x];
    rows = cut.rows(u);
    w = W1 + ((int64_t)e.e * F + r - x * F) * d;
    tiles = tiles_of(e.mask);
    const int some = __ffs(e.mask) - 1;
#pragma unroll
    for (int n = 0; n < NT; ++n) off[n] = (e.mask >> (8 * n + g) & 1 ? 8 * n + g : some) * d + 8 * t;
  }
};

// .. and here, where a column's sum runs over all experts, the row of zeros.
template <int NT, bool kTokens>
struct RowsOfHidden {
  MtCut cut;
  const __nv_bfloat16 *W2, *w;
  const MtShared* s;
  int F, K1, g, t, u, x, rows, zeros;
  int64_t dF;
  unsigned tiles;
  int off[NT];
  DG_DEV void start() {
    u = 0;
    x = -1;
    next();
  }
  DG_DEV void next() {
    if (++x > s->nact) {
      x = 0;
      ++u;
    }
    if (u >= cut.U) return;
    const MtExpert e = s->ex[x];
    if (!kTokens) {
      rows = cut.rows(u);
      w = W2 + (e.e * dF + cut.row(u) * F);
      return;
    }
    tiles = tiles_of(e.mask);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int m = 8 * n + g;
      off[n] = (e.mask >> m & 1 ? m * K1 + s->rank[x][m] : zeros) * 2 * F + 8 * t;
    }
  }
};

template <int NT>
__global__ void __launch_bounds__(kMtThreads, 1) moe_tokens_kernel(MtArgs a) {
  extern __shared__ __align__(16) char smem[];
  char* ring = smem + (threadIdx.x / 32) * kMtStages * kMtStage;
  float* red = reinterpret_cast<float*>(smem + kMtWarps * kMtStages * kMtStage);  // [units][warps][NT * 4][32]
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

  // A unit (32 rows at most) ends with each warp's part of its sums in `red`; the parts
  // are added, in order, after kBatch units or the last.  Then thread i * 32 + lane of a
  // unit's values has (row 16 r + g + 8 (i % 4 / 2), token 8 (i / 4 % NT) + 2 t + i % 2),
  // r = i / (4 NT).
  constexpr int kVals = 2 * NT * 4, kBatch = kMtRed / (kMtWarps * kVals * 128);
  auto add_parts = [&](int u0, int u1, const auto& put) {
    __syncthreads();
    for (int v = tid; v < (u1 - u0) * kVals * 32; v += kMtThreads) {
      const int u = u0 + v / (kVals * 32), at = v % (kVals * 32), i = at / 32;
      const float* from = red + (u % kBatch) * kMtWarps * kVals * 32 + at;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kMtWarps; ++w) sum += from[w * kVals * 32];
      put(u, 16 * (i / (4 * NT)) + g + 8 * (i % 4 / 2), 8 * (i / 4 % NT) + 2 * t + i % 2, sum);
    }
    __syncthreads();
  };

  // The engine of all phases.  A unit's sums run over segments (matrices of `pitch`
  // columns, KB blocks of 64 each); a warp takes every 16th block, over the borders of
  // segments and units.  It walks the segments with two cursors: one for the copies
  // (kMtStages - 1 blocks ahead), one for the tokens' values (a block ahead, in
  // registers, where they leave room).  A cursor gives the segment's first row w, rows,
  // unit u, the column tiles with tokens, the lane's offsets of the tokens' values, and
  // next().
  auto stream = [&](auto pc, auto bc, int KB, int pitch, int U, const __nv_bfloat16* values, auto pair, const auto& put) {
    constexpr bool kPair = decltype(pair)::value, kAhead = NT <= 2;
    constexpr int kB = kPair ? 2 : 1;
    int pk = warp, bk = warp, pslot = 0;
    auto settle = [&](auto& c, int& k) {
      while (k >= KB && c.u < U) {
        k -= KB;
        c.next();
      }
    };
    auto issue = [&]() {
      if (pc.u < U) {
        load_block(ring + pslot, pc.w + pk * 64, pitch, pc.rows, lane);
        pk += kMtWarps;
        settle(pc, pk);
      }
      cp_async_commit();
      pslot = pslot + kMtStage == kMtStages * kMtStage ? 0 : pslot + kMtStage;
    };
    uint4 b[NT][2][kB];
    auto load_b = [&](unsigned tiles, const int (&off)[NT], int k) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (NT == 1 || (tiles >> n & 1)) {
          const __nv_bfloat16* from = values + off[n] + k * 64 * kB;
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int q = 0; q < kB; ++q) b[n][p][q] = *reinterpret_cast<const uint4*>(from + (p * kB + q) * 32);
        }
    };
    settle(pc, pk);
    settle(bc, bk);
#pragma unroll 1
    for (int s0 = 0; s0 < kMtStages - 1; ++s0) issue();
    float acc[2][NT][4] = {};
    int u = 0, done = 0, slot = 0;
    auto flush_to = [&](int to) {  // units u .. to - 1 have all that this warp adds to them
#pragma unroll 1
      for (; u < to; ++u) {
        float* part = red + ((u % kBatch) * kMtWarps + warp) * kVals * 32 + lane;
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
          part[i * 32] = acc[i / (4 * NT)][i / 4 % NT][i % 4];
          acc[i / (4 * NT)][i / 4 % NT][i % 4] = 0.f;
        }
        if (u + 1 == U || (u + 1) % kBatch == 0) {
          add_parts(done, u + 1, put);
          done = u + 1;
        }
      }
    };
    flush_to(min(bc.u, U));
    if (kAhead && bc.u < U) load_b(bc.tiles, bc.off, bk);
#pragma unroll 1
    while (bc.u < U) {
      issue();
      cp_async_wait<kMtStages - 1>();
      const unsigned tiles = bc.tiles;
      if (!kAhead) load_b(tiles, bc.off, bk);
      bk += kMtWarps;
      settle(bc, bk);
      const char* from = ring + slot + lane * 16;
      slot = slot + kMtStage == kMtStages * kMtStage ? 0 : slot + kMtStage;
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 v = *reinterpret_cast<const uint4*>(from + (4 * r + p) * 512);
          const uint4 w = *reinterpret_cast<const uint4*>(from + (4 * r + 2 + p) * 512);
          const uint32_t A0[4] = {v.x, w.x, v.y, w.y}, A1[4] = {v.z, w.z, v.w, w.w};
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (NT == 1 || (tiles >> n & 1)) {
#pragma unroll
              for (int q = 0; q < kB; ++q) {
                mma_bf16_16816(acc[r][n], A0, b[n][p][q].x, b[n][p][q].y);
                mma_bf16_16816(acc[r][n], A1, b[n][p][q].z, b[n][p][q].w);
              }
            }
        }
      if (kAhead && bc.u < U) load_b(bc.tiles, bc.off, bk);
      flush_to(min(bc.u, U));
    }
    cp_async_wait<0>();
  };

  auto range = [&](int rows, int c) { return (int)((int64_t)rows * c / ctas); };
  auto store_hidden = [&](int m, int j, int f, float v) {
    const size_t at = ((size_t)m * K1 + j) * 2 * a.Fe + f / 32 * 64 + f % 32;
    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
    a.hid[at] = hi;
    a.hid[at + 32] = __float2bfloat16_rn(v - __bfloat162float(hi));
  };

  if (cta == 0)
    for (int i = tid; i < a.Fe / 4; i += kMtThreads)
      reinterpret_cast<uint4*>(a.hid + (size_t)a.M * K1 * 2 * a.Fe)[i] = make_uint4(0, 0, 0, 0);

  // ---- phase 0: the router's rows, then the shared expert's
  {
    const int n32 = (a.n_exp + kMtRows - 1) / kMtRows * kMtRows, R = n32 + a.Fe;
    const MtCut cut(range(R, cta), range(R, cta + 1), n32);
    RowsOfH0<NT> c;
    c.cut = cut;
    c.Wr = a.Wr;
    c.Ws = a.W1 + (int64_t)a.n_exp * a.Fe * a.d;
    c.border = n32;
    c.n_exp = a.n_exp;
    c.d = a.d;
    c.start(g, t, a.M);
    stream(c, c, KB1, a.d, cut.U, a.h, std::false_type{}, [&](int u, int row, int m, float v) {
      if (row >= cut.rows(u) || m >= a.M) return;
      row += cut.row(u);
      if (row < a.n_exp) a.logits[(size_t)m * a.n_exp + row] = v * s.inv[m];
      else if (row >= n32) store_hidden(m, a.top_k, row - n32, gelu(v * s.inv[m]));
    });
  }
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
      s.place[mye][m] = (uint8_t)lane;
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
      if (on) s.ex[n + __popc(b & ((1u << lane) - 1))] = MtExpert{e0 + lane, s.mask[e0 + lane]};
      n += __popc(b);
    }
    if (lane == 0) {
      s.nact = n;
      s.ex[n] = MtExpert{a.n_exp, all};
    }
  }
  __syncthreads();
  const int nact = s.nact;
  for (int i = tid; i < (nact + 1) * kMtMaxM; i += kMtThreads) {
    const int x = i / kMtMaxM, m = i % kMtMaxM;
    s.rank[x][m] = x < nact ? s.place[s.ex[x].e][m] : (uint8_t)a.top_k;
  }
  __syncthreads();

  // ---- phase 1: the chosen experts' hidden rows
  {
    const int R = nact * a.Fe, r0 = range(R, cta), r1 = range(R, cta + 1);
    const MtCut cut(r0, r1, min(r1, r0 / a.Fe * a.Fe + a.Fe));
    RowsOfH1<NT> c;
    c.cut = cut;
    c.W1 = a.W1;
    c.ex = s.ex;
    c.F = a.Fe;
    c.d = a.d;
    c.g = g;
    c.t = t;
    c.start();
    stream(c, c, KB1, a.d, cut.U, a.h, std::false_type{}, [&](int u, int row, int m, float v) {
      if (row >= cut.rows(u)) return;
      row += cut.row(u);
      const int x = row / a.Fe;
      if (!(s.ex[x].mask >> m & 1)) return;
      const int j = s.rank[x][m];
      store_hidden(m, j, row - x * a.Fe, s.gate[m][j] * gelu(v * s.inv[m]));
    });
  }
  if (!grid_barrier(a.bar, a.status, &s.stop)) return;

  // ---- phase 2: output columns, their sums over the experts' hidden values
  {
    const int r0 = range(a.d, cta), r1 = range(a.d, cta + 1);
    const MtCut cut(r0, r1, r1);
    auto cursor = [&](auto tokens) {
      RowsOfHidden<NT, decltype(tokens)::value> c;
      c.cut = cut;
      c.W2 = a.W2;
      c.s = &s;
      c.F = a.Fe;
      c.dF = (int64_t)a.d * a.Fe;
      c.K1 = K1;
      c.zeros = a.M * K1;
      c.g = g;
      c.t = t;
      c.start();
      return c;
    };
    stream(cursor(std::false_type{}), cursor(std::true_type{}), KB2, a.Fe, cut.U, a.hid, std::true_type{},
           [&](int u, int row, int m, float v) {
             if (row >= cut.rows(u) || m >= a.M) return;
             const int at = m * a.d + cut.row(u) + row;
             a.out[at] = __float2bfloat16_rn(__bfloat162float(a.h[at]) + v);
           });
  }
}

struct MtWs {
  size_t logits, hid, total;
};

MtWs mt_ws(int M, int n_exp, int top_k, int Fe) {
  MtWs w;
  size_t o = 256;  // status word, the barrier's two words
  w.logits = o;
  o = align_up(o + sizeof(float) * M * n_exp, 256);
  w.hid = o;
  o = align_up(o + 4 * ((size_t)M * (top_k + 1) + 1) * Fe, 256);
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
  const int smem = kMtWarps * kMtStages * kMtStage + kMtRed;
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
  a.hid = reinterpret_cast<__nv_bfloat16*>(base + w.hid);
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

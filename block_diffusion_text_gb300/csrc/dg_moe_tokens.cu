// A layer's whole mixture-of-experts block for a few tokens, in one launch:
//
//   x = RMSNorm(h), r = x Wr^T, e_j = the top_k experts of r, g = softmax of their r
//   out = h + sum_j g_j We2_ej GELU(We1_ej x) + We2_s GELU(We1_s x)
//
// The chosen experts' weights bound it: each matrix is read once for each eight of the
// tokens that chose it (from L2 after the first).  One persistent CTA per SM works
// through three phases with a barrier of the grid between them, as the data demands:
//   0  the router's logits
//   1  every CTA works the routing out for itself; the hidden rows of the chosen experts
//      and of the shared one
//   2  the output columns
// In each phase the rows of the weights that it needs are cut into equal ranges,
// one for each CTA, row by row, so that all SMs read the same number of bytes.
//
// Measured, 128 experts of 768 x 2816, top 8: one token 34 us (79 MB: 12 us at the copy
// rate; the router takes 4, routing 3, each barrier 2), 16 tokens 152 (723 MB, 108), 32
// tokens 211 (146).
//
// Warp MMAs, the weights as the 16-row operand, up to eight of the expert's own tokens as
// the columns: an expert with more of them comes several times.  (With a column for
// every token of the call, tiles of eight of them where one had chosen the expert,
// 32 tokens took 355 us at 128 experts of 768 x 2816.)
// x W^T is taken as (h W^T) / rms, so the tokens enter as the bf16 they are; the hidden
// values, which carry their gate (the second product is linear), as pairs of bf16 (16
// bits or more).  A warp's share of the products' inner dimension is a block of 64
// columns in turn; its own weights come through a ring of cp.async copies that only the
// lane that issued them reads, so nothing has to be waited for but the lane's own copies.
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
constexpr int kMtUnits = 16;    // units of a round
constexpr int kMtVals = 8;      // sums of a unit in a lane
constexpr int kMtPitch = kMtRows + 1;    // of a token's sums of an output unit
constexpr int kMtMaxM = 32;
constexpr int kMtMaxExp = 256, kMtMaxK = 16;
constexpr int kMtMaxSegs = kMtMaxExp + (kMtMaxM * kMtMaxK + kMtMaxM) / 8;

struct MtArgs {
  const __nv_bfloat16* h;                  // [M][d]
  __nv_bfloat16* out;                      // [M][d], may be h
  const __nv_bfloat16 *Wr, *W1, *W2;       // [n_exp][d], [n_exp + 1][Fe][d], [n_exp + 1][d][Fe]
  float* logits;                           // [M][n_exp], before the product with 1 / rms
  __nv_bfloat16* hid;                      // [M (top_k + 1)][Fe / 32][2][32]: gate GELU(x We1^T), the values as
                                           // bf16 and what that leaves
  int* idx;                                // [M][top_k] or null
  float* gate;                             // [M][top_k] or null
  int* status;
  unsigned *arrivals, *rounds;             // of the grid's barrier
  int M, d, Fe, n_exp, top_k;
  float eps;
};

// An expert with up to eight of its tokens
struct MtSeg {
  int e, n;
  uint8_t tok[8], rank[8];                 // the tokens, and the expert's place among theirs
};

struct MtShared {
  float inv[kMtMaxM];
  float squares[kMtMaxM][kMtWarps];
  float gate[kMtMaxM][kMtMaxK];
  unsigned mask[kMtMaxExp + 32];           // tokens of every expert, all for the shared one, and zeros
  uint8_t sel[kMtMaxM][kMtMaxK];           // a token's experts in rank order
  uint16_t pos[kMtMaxExp + 1];             // an expert's first place in seg
  MtSeg seg[kMtMaxSegs];                   // of the experts with tokens, ascending, and the shared one's
  int nseg;
  int stop;
};

// One arrival at the grid's barrier; the last of a round begins the next.  The count wraps
// to zero by itself.
DG_DEV bool grid_arrive(unsigned* arrivals, unsigned* rounds) {
  __threadfence();
  if (atomicInc(arrivals, gridDim.x - 1) != gridDim.x - 1) return false;
  __threadfence();
  atomicAdd(rounds, 1u);
  return true;
}

// All CTAs of the grid are here (the launch is cooperative).  Thread 0 arrives for its
// CTA.  Arrivals and rounds lie in memory lines of their own: a line that is polled while
// others write to it goes back and forth between the dies (flags of the CTAs side by side
// took 6 us).  Bounded: false, with the status word set, if the others do not come.  A
// CTA that gives up arrives all the same at the barriers that it will not come to: every
// launch makes two rounds of arrivals, so the next one finds the count at zero.
DG_DEV bool grid_barrier(unsigned* arrivals, unsigned* rounds, int* status, int* stop) {
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned round;
    asm volatile("ld.relaxed.gpu.u32 %0, [%1];" : "=r"(round) : "l"(rounds) : "memory");
    if (!grid_arrive(arrivals, rounds)) {
      uint64_t t0 = 0;
      for (unsigned i = 0;; ++i) {
        unsigned now;
        asm volatile("ld.relaxed.gpu.u32 %0, [%1];" : "=r"(now) : "l"(rounds) : "memory");
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

// L2 takes 256 bytes about them: a row's next block is there when its turn comes, and a
// page of the memory is opened half as often (16 tokens of 128 experts of 768 x 2816: 152
// us, 166 without; blocks of 128 columns 159, prefetches of whole pieces of a row 174).
DG_DEV void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

DG_DEV float gelu(float x) { return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f)); }

// Stage of a ring: the lane's pieces of rows g, g + 8, g + 16 and g + 24, halves 0 and
// 1 of the 64 columns.  Rows at or past `rows` are not copied: what their products
// hold is not used.
DG_DEV void load_block(char* slot, const __nv_bfloat16* src, int pitch, int rows, int lane) {
#pragma unroll
  for (int r = 0; r < kMtRows / 8; ++r)
    if (lane / 4 + 8 * r < rows) {
#pragma unroll
      for (int p = 0; p < 2; ++p) cp_async16(slot + ((r * 2 + p) * 32 + lane) * 16, src + 8 * r * pitch + 32 * p);
    }
}

// Rows [r0, r1) cut into units of 32 rows at most, from r0 to the border rb (a
// matrix's end) and from there on.  (Further matrices begin at multiples of 32 from
// there: their rows are multiples of 128.)
struct MtCut {
  int r0, rb, r1, U0, U;
  DG_DEV MtCut(int first, int end, int border) : r0(first), r1(end) {
    rb = border > first && border < end ? border : end;
    U0 = (rb - r0 + kMtRows - 1) / kMtRows;
    U = U0 + (r1 - rb + kMtRows - 1) / kMtRows;
  }
  DG_DEV int row(int u) const { return u < U0 ? r0 + kMtRows * u : rb + kMtRows * (u - U0); }
  DG_DEV int rows(int u) const { return min(kMtRows, (u < U0 ? rb : r1) - row(u)); }
};

__global__ void __launch_bounds__(kMtThreads, 1) moe_tokens_kernel(MtArgs a) {
  extern __shared__ __align__(16) char smem[];
  char* ring = smem + (threadIdx.x / 32) * kMtStages * kMtStage;
  // sums: [warps + units - 1][kMtVals][32], or [warps][M][kMtPitch] of an output unit
  float* red = reinterpret_cast<float*>(smem + kMtWarps * kMtStages * kMtStage);
  __shared__ MtShared s;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int K1 = a.top_k + 1, KB1 = a.d / 64, KB2 = a.Fe / 64;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (tid == 0) s.stop = 0;

  // 1 / rms of every token, for this CTA's own use: 16 / M warps to a token
  auto norms = [&]() {
    const int per = a.M >= kMtWarps ? 1 : kMtWarps / a.M, m0 = warp / per, part = warp % per, n8 = a.d / 8;
    for (int m = m0; m < a.M; m += kMtWarps / per) {
      float sum = 0.f;
      const uint4* src = reinterpret_cast<const uint4*>(a.h + (size_t)m * a.d);
      for (int i0 = part * 32 + lane; i0 < n8; i0 += per * 128) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i0 + k * per * 32 < n8 ? src[i0 + k * per * 32] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = __uint_as_float(w[j] << 16), y = __uint_as_float(w[j] & 0xffff0000u);
            sum += x * x + y * y;
          }
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) s.squares[m][part] = sum;
    }
    __syncthreads();
    if (tid < a.M) {
      float sum = 0.f;
      for (int p = 0; p < per; ++p) sum += s.squares[tid][p];
      // (beyond fp32 the row would come out as zeros, and the routing as that of zeros)
      if (!(sum <= FLT_MAX) && cta == 0) atomicCAS(a.status, 0, kStatusValue);
      s.inv[tid] = 1.0f / sqrtf(sum / (float)a.d + a.eps);
    }
    // (read after the barrier before the units' sums)
  };

  // The engine of all phases.  Work comes in rounds of some segments, matrices of KB
  // blocks of 64 columns and up to 32 rows; a round's blocks, in that order, are dealt to
  // the warps in equal shares, so a warp has parts of one segment or of several: a task
  // each.  The parts of a segment's sums are added up, in order, when the round ends,
  // and given to put(round, segment, row, column, sum); with kOne the round is one unit of
  // output rows, to which all segments add: a warp adds its parts up for their tokens,
  // and put gets (round, 0, row, token, sum).
  // The first copies are on their way before gate() is passed (the weights wait for
  // nobody).  They run ahead over all borders, the tokens' values a block ahead within a
  // task.
  auto stream = [&](int F, const auto& segments, int KB, int pitch, auto one, const auto& seg_w, const auto& seg_b,
                    const __nv_bfloat16* values, auto pair, const auto& gate, const auto& meanwhile, const auto& put) {
    constexpr bool kOne = decltype(one)::value;
    constexpr int kB = decltype(pair)::value ? 2 : 1;
    // of n blocks; where there are fewer blocks than warps, one each for the first warps
    auto share = [&](int n, int* first, int* end) {
      const int W = min(n, kMtWarps);
      *first = warp < W ? n * warp / W : 0;
      *end = warp < W ? n * (warp + 1) / W : 0;
    };
    int pf = -1, pi = 0, pe = 0, pn = 0, prows = 0, pslot = 0;
    const __nv_bfloat16* pw = nullptr;
    auto issue = [&]() {
      while (pn == 0 && pf < F) {  // the next task
        if (pi == pe) {
          if (++pf == F) break;
          const int total = segments(pf) * KB;
          share(total, &pi, &pe);
          continue;
        }
        const int seg = pi / KB, kb = pi - seg * KB;
        seg_w(pf, seg, &pw, &prows);
        pw += g * pitch + kb * 64 + 8 * t;
        pn = min(KB - kb, pe - pi);
        pi += pn;
      }
      if (pn > 0) {
        load_block(ring + pslot, pw, pitch, prows, lane);
        pw += 64;
        --pn;
      }
      cp_async_commit();
      pslot = pslot + kMtStage == kMtStages * kMtStage ? 0 : pslot + kMtStage;
    };
#pragma unroll 1
    for (int s0 = 0; s0 < kMtStages; ++s0) issue();
    float* own = red + warp * a.M * kMtPitch;
    auto clear = [&]() {
      for (int i = lane; i < a.M * kMtPitch; i += 32) own[i] = 0.f;
      __syncwarp();
    };
    if (kOne) clear();
    if (!gate()) {
      cp_async_wait<0>();
      return false;
    }
    int slot = 0;
#pragma unroll 1
    for (int f = 0; f < F; ++f) {
      const int segs = segments(f), total = segs * KB;
      int i, end;
      share(total, &i, &end);
#pragma unroll 1
      while (i < end) {
        const int seg = i / KB, kb = i - seg * KB;
        int nb = min(KB - kb, end - i);
        i += nb;
        const __nv_bfloat16* from = values + seg_b(f, seg) + kb * 64 * kB;
        float acc[2][4] = {};
        uint4 b[2][kB];
        auto load_b = [&]() {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int q = 0; q < kB; ++q) b[p][q] = *reinterpret_cast<const uint4*>(from + (p * kB + q) * 32);
          from += 64 * kB;
        };
        load_b();
#pragma unroll 1
        for (; nb > 0; --nb) {
          cp_async_wait<kMtStages - 1>();
          const char* at = ring + slot + lane * 16;
          slot = slot + kMtStage == kMtStages * kMtStage ? 0 : slot + kMtStage;
          uint32_t A[2][2][2][4];
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint4 v = *reinterpret_cast<const uint4*>(at + (4 * r + p) * 512);
              const uint4 w = *reinterpret_cast<const uint4*>(at + (4 * r + 2 + p) * 512);
              A[p][r][0][0] = v.x, A[p][r][0][1] = w.x, A[p][r][0][2] = v.y, A[p][r][0][3] = w.y;
              A[p][r][1][0] = v.z, A[p][r][1][1] = w.z, A[p][r][1][2] = v.w, A[p][r][1][3] = w.w;
            }
          issue();  // into the slot just read
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int q = 0; q < kB; ++q)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                mma_bf16_16816(acc[r], A[p][r][0], b[p][q].x, b[p][q].y);
                mma_bf16_16816(acc[r], A[p][r][1], b[p][q].z, b[p][q].w);
              }
          if (nb > 1) load_b();
        }
        // a lane's value v: row 16 (v / 4) + g + 8 (v % 4 / 2), column 2 t + v % 2
        if (kOne) {
          const MtSeg& x = s.seg[seg];
#pragma unroll
          for (int v = 0; v < kMtVals; ++v) {
            const int col = 2 * t + v % 2;
            if (col < x.n) own[x.tok[col] * kMtPitch + 16 * (v / 4) + g + 8 * (v % 4 / 2)] += acc[v / 4][v % 4];
          }
          __syncwarp();
        } else {
          float* part = red + (warp + seg) * kMtVals * 32 + lane;
#pragma unroll
          for (int v = 0; v < kMtVals; ++v) part[v * 32] = acc[v / 4][v % 4];
        }
      }
      if (f == 0) meanwhile();
      __syncthreads();
      if (kOne) {
        for (int v = tid; v < a.M * kMtRows; v += kMtThreads) {
          const float* src = red + v / kMtRows * kMtPitch + v % kMtRows;
          float sum = 0.f;
#pragma unroll 4
          for (int w = 0; w < kMtWarps; ++w) sum += src[w * a.M * kMtPitch];
          put(f, 0, v % kMtRows, v / kMtRows, sum);
        }
      } else {
        // the parts of a segment are those of the warps from the owner of its first block
        // to that of its last
        const int W = min(total, kMtWarps);
        for (int v = tid; v < segs * kMtVals * 32; v += kMtThreads) {
          const int u = v / (kMtVals * 32), i = v / 32 % kMtVals;
          const int w0 = ((u * KB + 1) * W - 1) / total, w1 = ((u + 1) * KB * W - 1) / total;
          const float* src = red + (u * kMtVals + i) * 32 + lane;
          float sum = 0.f;
#pragma unroll 4
          for (int w = w0; w <= w1; ++w) sum += src[w * kMtVals * 32];
          put(f, u, 16 * (i / 4) + g + 8 * (i % 4 / 2), 2 * t + i % 2, sum);
        }
      }
      __syncthreads();
      if (kOne) clear();
    }
    if (F == 0) meanwhile();
    cp_async_wait<0>();
    return true;
  };
  auto go = [] { return true; };
  auto rounds = [](const MtCut& cut) { return (cut.U + kMtUnits - 1) / kMtUnits; };
  auto units = [](const MtCut& cut, int f) { return min(kMtUnits, cut.U - f * kMtUnits); };
  auto range = [&](int rows, int c) { return (int)((int64_t)rows * c / ctas); };
  auto store_hidden = [&](int m, int j, int f, float v) {
    const size_t at = ((size_t)m * K1 + j) * 2 * a.Fe + f / 32 * 64 + f % 32;
    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
    a.hid[at] = hi;
    a.hid[at + 32] = __float2bfloat16_rn(v - __bfloat162float(hi));
  };

  for (int e = tid; e < kMtMaxExp + 32; e += kMtThreads) s.mask[e] = e == a.n_exp ? ~0u >> (32 - a.M) : 0u;

  // ---- phase 0: the router's rows, for each eight tokens (a range of rows is shorter than
  // the matrix, so it meets no second border)
  {
    const int R = (a.M + 7) / 8 * a.n_exp, r0 = range(R, cta), r1 = range(R, cta + 1);
    const MtCut cut(r0, r1, min(r1, r0 / a.n_exp * a.n_exp + a.n_exp));
    stream(rounds(cut), [&](int f) { return units(cut, f); }, KB1, a.d, std::false_type{},
           [&](int f, int u, const __nv_bfloat16** w, int* rows) {
             u += f * kMtUnits;
             *rows = cut.rows(u);
             *w = a.Wr + (int64_t)(cut.row(u) % a.n_exp) * a.d;
           },
           // columns past the last token repeat it
           [&](int f, int u) { return min(cut.row(u + f * kMtUnits) / a.n_exp * 8 + g, a.M - 1) * a.d + 8 * t; },
           a.h, std::false_type{}, go, norms, [&](int f, int u, int row, int col, float v) {
             u += f * kMtUnits;
             const int r = cut.row(u) + row, m = cut.row(u) / a.n_exp * 8 + col;
             if (row < cut.rows(u) && m < a.M) a.logits[(size_t)m * a.n_exp + r % a.n_exp] = v;
           });
  }
  if (!grid_barrier(a.arrivals, a.rounds, a.status, &s.stop)) {
    if (tid == 0) grid_arrive(a.arrivals, a.rounds);  // for the second barrier
    return;
  }

  // ---- the routing.  Keys in the order of the logits, 0 for NaN; equal ones by index.
  auto key_of = [&](float l) { return l == l ? float_key(l == 0.f ? 0.f : l) : 0u; };
  auto chosen = [&](int m, int k, int e, float gt) {
    s.gate[m][k] = gt;
    s.sel[m][k] = (uint8_t)e;
    atomicOr(&s.mask[e], 1u << m);
    if (cta == 0) {
      if (a.idx) a.idx[(size_t)m * a.top_k + k] = e;
      if (a.gate) a.gate[(size_t)m * a.top_k + k] = gt;
    }
  };
  if (a.M * a.n_exp <= kMtThreads) {
    // few logits: each is ranked by a team of threads that compares it with all others
    // (0.9 us; a warp that picks the largest one after the other takes 2.6)
    unsigned* keys = reinterpret_cast<unsigned*>(red);  // [M][n_exp]
    const int pairs = a.M * a.n_exp;
    float mine = 0.f;
    if (tid < pairs) {
      const int m = tid / a.n_exp;
      mine = __ldcg(a.logits + tid) * s.inv[m];
      if (!(fabsf(mine) <= FLT_MAX) && cta == 0) atomicCAS(a.status, 0, kStatusValue);
      keys[tid] = key_of(mine);
      red[kMtThreads + tid] = mine;
    }
    __syncthreads();
    int team = 1;
    while (team < 32 && pairs * team * 2 <= kMtThreads) team *= 2;
    const int pair = tid / team, m = pair / a.n_exp, e = pair - m * a.n_exp, mate = tid % team;
    int rank = 0;
    if (pair < pairs) {
      const unsigned* of = keys + m * a.n_exp;
      const unsigned key = of[e];
      for (int o = mate; o < a.n_exp; o += team) rank += of[o] > key || (of[o] == key && o < e);
    }
    for (int o = 1; o < team; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    float* top = red + 2 * kMtThreads;  // [M][top_k] logits in rank order
    if (pair < pairs && mate == 0 && rank < a.top_k) {
      top[m * a.top_k + rank] = keys[pair] ? red[kMtThreads + pair] : -FLT_MAX;
      s.sel[m][rank] = (uint8_t)e;
    }
    __syncthreads();
    if (tid < a.M * a.top_k) {
      const int row = tid / a.top_k, k = tid - row * a.top_k;
      const float* v = top + row * a.top_k;
      float Z = 0.f;
      for (int j = 0; j < a.top_k; ++j) Z += expf(v[j] - v[0]);
      chosen(row, k, s.sel[row][k], expf(v[k] - v[0]) / Z);
    }
  } else {
    // one warp for each token, a lane holding experts lane, lane + 32, ..
    for (int m = warp; m < a.M; m += kMtWarps) {
      float l[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) l[j] = lane + 32 * j < a.n_exp ? __ldcg(a.logits + (size_t)m * a.n_exp + lane + 32 * j) : 0.f;
      // keys in the order of the values; 0: no expert, taken, or NaN
      unsigned key[8];
      bool wrong = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        l[j] *= s.inv[m];
        const bool there = lane + 32 * j < a.n_exp;
        wrong |= there && !(fabsf(l[j]) <= FLT_MAX);
        key[j] = there ? key_of(l[j]) : 0u;
      }
      if (__any_sync(0xffffffffu, wrong) && lane == 0 && cta == 0) atomicCAS(a.status, 0, kStatusValue);
      float top = 0.f, Z = 0.f, mine = 0.f;
      int mye = 0;
      unsigned taken = 0;
#pragma unroll 1
      for (int k = 0; k < a.top_k; ++k) {
        unsigned best = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) best = max(best, key[j]);
        best = __reduce_max_sync(0xffffffffu, best);
        int first = INT_MAX;  // the lowest one with that value (of value 0: not taken)
#pragma unroll
        for (int j = 7; j >= 0; --j)
          if (key[j] == best && !(taken >> j & 1) && lane + 32 * j < a.n_exp) first = lane + 32 * j;
        const int be = (int)__reduce_min_sync(0xffffffffu, (unsigned)first);
        if ((be & 31) == lane) {
          taken |= 1u << (be >> 5);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j == be >> 5) key[j] = 0u;
        }
        const float bv = best ? key_float(best) : -FLT_MAX;
        if (k == 0) top = bv;
        Z += expf(bv - top);
        if (lane == k) {
          mine = bv;
          mye = be;
        }
      }
      if (lane < a.top_k) chosen(m, lane, mye, expf(mine - top) / Z);
    }
  }
  __syncthreads();
  if (warp == 0) {
    int n = 0;
#pragma unroll 1
    for (int e = lane; e - lane <= a.n_exp; e += 32) {
      const int tokens = __popc(s.mask[e]);
      int first = n;
#pragma unroll 1
      for (int j = 0; j < a.M; j += 8) {
        const unsigned some = __ballot_sync(0xffffffffu, tokens > j);
        first += __popc(some & ((1u << lane) - 1));
        n += __popc(some);
      }
      if (tokens) s.pos[e] = (uint16_t)first;
#pragma unroll 1
      for (int j = 0; j < tokens; j += 8, ++first) {
        s.seg[first].e = e;
        s.seg[first].n = min(8, tokens - j);
      }
    }
    if (lane == 0) s.nseg = n;
  }
  __syncthreads();
  const int nseg = s.nseg;
  for (int i = tid; i < a.M * K1; i += kMtThreads) {
    const int m = i / K1, j = i - m * K1;
    const int e = j < a.top_k ? s.sel[m][j] : a.n_exp, at = __popc(s.mask[e] & ((1u << m) - 1));
    MtSeg& x = s.seg[s.pos[e] + at / 8];
    x.tok[at % 8] = (uint8_t)m;
    x.rank[at % 8] = (uint8_t)j;
  }
  __syncthreads();

  // ---- phase 1: the hidden rows of the chosen experts, then of the shared one
  {
    const int R = nseg * a.Fe, r0 = range(R, cta), r1 = range(R, cta + 1);
    const MtCut cut(r0, r1, min(r1, r0 / a.Fe * a.Fe + a.Fe));
    stream(rounds(cut), [&](int f) { return units(cut, f); }, KB1, a.d, std::false_type{},
           [&](int f, int u, const __nv_bfloat16** w, int* rows) {
             const int r = cut.row(u + f * kMtUnits), x = r / a.Fe;
             *rows = cut.rows(u + f * kMtUnits);
             *w = a.W1 + ((int64_t)s.seg[x].e * a.Fe + r - x * a.Fe) * a.d;
           },
           [&](int f, int u) {  // (columns without a token repeat the first)
             const MtSeg& x = s.seg[cut.row(u + f * kMtUnits) / a.Fe];
             return x.tok[g < x.n ? g : 0] * a.d + 8 * t;
           },
           a.h, std::false_type{}, go, [] {}, [&](int f, int u, int row, int col, float v) {
             u += f * kMtUnits;
             if (row >= cut.rows(u)) return;
             row += cut.row(u);
             const MtSeg& x = s.seg[row / a.Fe];
             if (col >= x.n) return;
             const int m = x.tok[col], j = x.rank[col];
             store_hidden(m, j, row % a.Fe, (j < a.top_k ? s.gate[m][j] : 1.0f) * gelu(v * s.inv[m]));
           });
  }

  // ---- phase 2: output columns, their sums over the experts' hidden values
  {
    const int r0 = range(a.d, cta), r1 = range(a.d, cta + 1);
    const MtCut cut(r0, r1, r1);
    stream(cut.U, [&](int) { return nseg; }, KB2, a.Fe, std::true_type{},
           [&](int f, int x, const __nv_bfloat16** w, int* rows) {
             *rows = cut.rows(f);
             *w = a.W2 + ((int64_t)s.seg[x].e * a.d + cut.row(f)) * a.Fe;
           },
           [&](int, int k) {
             const MtSeg& x = s.seg[k];
             const int col = g < x.n ? g : 0;
             return (x.tok[col] * K1 + x.rank[col]) * 2 * a.Fe + 8 * t;
           },
           a.hid, std::true_type{}, [&] { return grid_barrier(a.arrivals, a.rounds, a.status, &s.stop); }, [] {},
           [&](int u, int, int row, int m, float v) {
             if (row >= cut.rows(u)) return;
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
  size_t o = 768;  // status word, the barrier's two lines
  w.logits = o;
  o = align_up(o + sizeof(float) * M * n_exp, 256);
  w.hid = o;
  o = align_up(o + 4 * (size_t)M * (top_k + 1) * Fe, 256);
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

cudaError_t launch(const MtArgs& a, int sms, cudaStream_t st) {
  const int sums = (kMtWarps + kMtUnits - 1) * kMtVals * 32, tokens = kMtWarps * a.M * kMtPitch;
  constexpr int most = kMtWarps * (kMtStages * kMtStage + kMtMaxM * kMtPitch * (int)sizeof(float));
  const int smem = kMtWarps * kMtStages * kMtStage + (sums > tokens ? sums : tokens) * (int)sizeof(float);
  cudaError_t e = set_smem_once<moe_tokens_kernel>(most);
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
  return cudaLaunchKernelEx(&cfg, moe_tokens_kernel, a);
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
  a.arrivals = reinterpret_cast<unsigned*>(base + 256);
  a.rounds = reinterpret_cast<unsigned*>(base + 512);
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
  const cudaError_t e = launch(a, sms, st);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

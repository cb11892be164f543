// Tokens from logits with temperature, top-k, top-p and min-p, by given random
// numbers.
//
// A row's tokens are ordered by value, the lower index first where two are equal, and
// weigh w = exp((l - max) / T).  What is kept is a leading run of that order, cut at
// the tightest of: the first k; the smallest run that holds top_p of what top-k left;
// w >= min_p.  The token drawn is the first, by index, at which the running sum of the
// kept weights passes u times their total.
//
// Two decisions compare sums over the vocabulary with a border, so the sums are whole
// numbers: a weight is a fixed-point number (30 bits and an exponent, on the scale of
// the row's largest), sums are 64 bits wide and exact, whatever order the atomics add
// them in, and a border between tokens is where the exact arithmetic has it but for
// the weights' own 2^-29.
//
// A cluster of CTAs takes a row: each holds a slice in shared memory, read once from
// global memory (what bounds the call), and the passes over it are on chip.  A cut is
// found by histograms over the slices, summed through the cluster's shared memory: a
// first one linear in the value below the maximum, further ones over the bits of the
// values in the bin that holds the border, until a bin is a single value.
#include <cfloat>
#include <climits>
#include <cmath>

#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kSpThreads = 512;
constexpr int kSpWarps = kSpThreads / 32;
constexpr int kSpBins = 2048;
constexpr int kSpMaxV = 1 << 20;
constexpr int kSpMaxCluster = 16;
constexpr int kSpTable = 64;                  // 2^(j / 64)
constexpr int kSpTop = 43;                    // a weight of the row's scale is 2^43: 2^20 of them stay below 2^63
constexpr float kSpUnit = 32.0f;              // bins of the first histogram to a factor of two in weight
constexpr int kSpHeld = 45056;                // most values of a slice held in shared memory

struct SpArgs {
  const void* logits;  // fp32 or bf16 [R][ld]
  const float *u, *temperature, *top_p, *min_p;
  const int* top_k;
  int32_t *token, *kept;
  float* logprob;
  int64_t ld;
  int R, V, slice, held, bf16;
  float temperature_all, top_p_all, min_p_all;
  int top_k_all;
};

struct SpTables {
  uint32_t t[kSpTable];  // 2^29 2^(j / 64), rounded
};

// What the CTAs of a cluster tell each other: a slot for each, so that a sum is taken
// in the same order everywhere.
struct SpBoard {
  unsigned long long a[kSpMaxCluster];
  unsigned long long b[kSpMaxCluster];
};

// A row's scale: x = (l - base) log2(e) / T.  base is zero, or where max / T is large
// the maximum: a difference to it that matters is exact then.
struct SpScale {
  float c, clo;    // log2(e) / T
  float base;
  int nref;        // weights are relative to 2^nref, above the largest
};

struct SpShared {
  unsigned count[kSpBins];
  unsigned lo[kSpBins], hi[kSpBins];      // masses, 64 bits in two words
  unsigned long long sum[kSpBins];        // this CTA's part of the bins, summed over the cluster (masses or counts)
  uint2 pow2[kSpTable];                   // the table entry as an integer and as a float
  SpBoard board[4];
  unsigned long long warp_a[kSpWarps], warp_b[kSpWarps];
  unsigned long long found_above;
  int found_bin;
  unsigned found_flag;
  SpScale scale;
  unsigned floor_key;
};

DG_DEV unsigned ld_cluster_u32(uint32_t a) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
DG_DEV void st_cluster_u64(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// The weight of a value, 2^(x - nref + 43) rounded down to a whole number.  x = l c is
// taken as a sum of two floats, so that r = x - k / 64 keeps all its bits; 2^(k / 64)
// comes from the table and 2^r - 1 from three terms of its series (the fourth is
// below 2^-34); their product is added in units of 2^-29 of the table's scale.
DG_DEV unsigned long long weight_of(float v, const SpScale& s, const uint2* pow2) {
  const float l = v - s.base;
  float x = l * s.c;
  float e = fmaf(l, s.c, -x);
  e = fmaf(l, s.clo, e);
  // values far below the largest weigh nothing (and x may be -inf)
  if (!(x > (float)(s.nref - 64))) return 0ull;
  const float kf = rintf(x * 64.0f);
  const int k = (int)kf;
  const float r = fmaf(kf, -0.015625f, x) + e;
  const float q = r * fmaf(r, fmaf(r, 0.05550410866f, 0.2402265070f), 0.6931471806f);
  const uint2 t = pow2[k & (kSpTable - 1)];
  const unsigned m = t.x + (unsigned)__float2int_rn(__uint_as_float(t.y) * q);
  const int sh = s.nref - (k >> 6);  // 0 .. 64
  return sh < 44 ? ((unsigned long long)m << (kSpTop - 29)) >> sh : 0ull;
}

DG_DEV unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of two numbers over the CTA, in every thread.
DG_DEV void cta_sum(SpShared& s, unsigned long long& a, unsigned long long& b) {
  a = warp_sum(a);
  b = warp_sum(b);
  __syncthreads();
  if (threadIdx.x % 32 == 0) {
    s.warp_a[threadIdx.x / 32] = a;
    s.warp_b[threadIdx.x / 32] = b;
  }
  __syncthreads();
  a = b = 0;
  for (int w = 0; w < kSpWarps; ++w) {
    a += s.warp_a[w];
    b += s.warp_b[w];
  }
}

// Puts this CTA's numbers on every CTA's board `which` and waits for the others'.
// A board is used again after another exchange at the earliest.
DG_DEV void exchange(SpShared& s, int which, unsigned long long a, unsigned long long b, uint32_t rank, uint32_t ctas) {
  if (threadIdx.x < ctas) {
    st_cluster_u64(cluster_addr(&s.board[which].a[rank], threadIdx.x), a);
    st_cluster_u64(cluster_addr(&s.board[which].b[rank], threadIdx.x), b);
  }
  cluster_sync();
}

// floor(x f) and ceil(x f) for a fraction 0 <= f < 1 (below 2^-40 bits are dropped).
DG_DEV unsigned long long fraction(float f) { return (unsigned long long)(f * 18446744073709551616.0f); }

DG_DEV float value_at(const SpArgs& a, const float* held, const char* row, int base, int i) {
  if (i < a.held) return held[i];
  return a.bf16 ? __uint_as_float((unsigned)reinterpret_cast<const uint16_t*>(row)[base + i] << 16)
                : reinterpret_cast<const float*>(row)[base + i];
}

// The order of values; -0 and 0 are equal.
DG_DEV unsigned key_of(float v) { return float_key(v == 0.f ? 0.f : v); }

// The cut of a leading run: values above `key` are in, and of those equal to it the
// first `ties` by index.
struct SpCut {
  unsigned key;
  unsigned long long ties;
};

__global__ void __launch_bounds__(kSpThreads) sample_kernel(SpArgs a, SpTables tables) {
  extern __shared__ float held[];
  __shared__ SpShared s;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t ctas = gridDim.y, rank = cluster_ctarank();
  const int row = blockIdx.x;
  const char* src = static_cast<const char*>(a.logits) + (size_t)row * a.ld * (a.bf16 ? 2 : 4);
  const int base = (int)rank * a.slice;
  const int n = max(0, min(a.slice, a.V - base));  // this CTA's values
  pdl_wait();
  for (int i = tid; i < kSpTable; i += kSpThreads) s.pow2[i] = make_uint2(tables.t[i], __float_as_uint((float)tables.t[i]));

  const float T = a.temperature ? a.temperature[row] : a.temperature_all;
  const float top_p = a.top_p ? a.top_p[row] : a.top_p_all, min_p = a.min_p ? a.min_p[row] : a.min_p_all;
  const int top_k = a.top_k ? a.top_k[row] : a.top_k_all;
  const float u = a.u[row];
  bool bad = !(T >= 0.f && T <= FLT_MAX) || !(top_p >= 0.f) || !(min_p >= 0.f && min_p <= 1.f) || top_k < 0 || !(u >= 0.f && u < 1.f);

  // ---- the slice, its largest value, its finite ones
  unsigned mkey = 0, fin = 0, wrong = 0;
  for (int i = tid; i < n; i += kSpThreads) {
    const float v = a.bf16 ? __uint_as_float((unsigned)reinterpret_cast<const uint16_t*>(src)[base + i] << 16)
                           : __ldcs(reinterpret_cast<const float*>(src) + base + i);
    if (i < a.held) held[i] = v;
    if (!(v <= FLT_MAX)) wrong = 1;
    else if (v >= -FLT_MAX) {
      ++fin;
      mkey = max(mkey, key_of(v));
    }
  }
  mkey = __reduce_max_sync(0xffffffffu, mkey);
  wrong = __reduce_max_sync(0xffffffffu, wrong);
  unsigned long long pa = fin, pb = 0;
  cta_sum(s, pa, pb);
  const unsigned long long fin_here = pa;
  __syncthreads();
  if (lane == 0) s.warp_a[warp] = ((unsigned long long)wrong << 32) | mkey;
  __syncthreads();
  unsigned long long mw = 0;
  for (int w = 0; w < kSpWarps; ++w) {
    const unsigned long long x = s.warp_a[w];
    mw = ((mw | x) >> 32 << 32) | max((unsigned)mw, (unsigned)x);
  }
  cluster_sync();  // every CTA of the cluster runs before another writes to it
  exchange(s, 0, mw, fin_here, rank, ctas);
  unsigned long long finite = 0;
  mkey = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    mkey = max(mkey, (unsigned)s.board[0].a[c]);
    bad |= (s.board[0].a[c] >> 32) != 0;
    finite += s.board[0].b[c];
  }
  bad |= finite == 0;
  const float m = bad ? 0.f : key_float(mkey);

  // Everything from here on is the same in all CTAs of the cluster but for their
  // slices, so that they come to every exchange together.
  SpCut cut{0u, ~0ull};       // all
  unsigned floor_key = 1u;    // min_p's: values at least this (finite ones)
  const bool greedy = T < 5.421010862427522e-20f || top_k == 1;  // 2^-64
  SpScale sc{0.f, 0.f, 0.f, 0};
  unsigned long long kept = finite, total = 0;
  if (!bad) {
    if (greedy) {
      cut.key = mkey;
      cut.ties = 1;
      kept = 1;
    } else {
      if (tid == 0) {  // in 64 bits, which few units compute
        const double c = 1.4426950408889634074 / (double)T, xm = (double)m * c;
        const float base_v = fabs(xm) > 16384.0 ? m : 0.f;
        s.scale = SpScale{(float)c, (float)(c - (double)(float)c), base_v, (int)ceil(base_v != 0.f ? 0.0 : xm) + 1};
        unsigned fk = 1u;
        if (min_p > 0.f) {
          // w >= min_p where l >= max + T ln(min_p): the first float at or above that border
          const double border = (double)m + (double)T * log((double)min_p);
          if (border >= -(double)FLT_MAX) {
            const float f = (float)border;
            fk = min(key_of(f) + ((double)f < border ? 1u : 0u), mkey);
          }
        }
        s.floor_key = fk;
      }
      __syncthreads();
      sc = s.scale;
      floor_key = s.floor_key;
    }
  }

  // One cut: the smallest leading run, within `cut` as it is, whose count or mass
  // reaches `target`.  False: the histogram's range does not reach so far.
  auto bin1 = [&](float v) { return (int)fminf((m - v) * (sc.c * kSpUnit), (float)(kSpBins - 1)); };
  // place of value i of this slice among those equal to the cut's key, in the whole row
  unsigned long long ties_before = 0;
  auto find_cut = [&](bool mass, unsigned long long target, const SpCut in) {
    unsigned khi = mkey, klo = 0;
    int shift = -1, want = -1;         // first level: linear in the value
    unsigned long long above = 0;      // what lies above the bin under search
    SpCut out{0u, ~0ull};
    for (int level = 0;; ++level) {
      for (int i = tid; i < kSpBins; i += kSpThreads) s.count[i] = s.lo[i] = s.hi[i] = 0u;
      __syncthreads();
      for (int i = tid; i < n; i += kSpThreads) {
        const float v = value_at(a, held, src, base, i);
        if (!(v >= -FLT_MAX)) continue;
        const unsigned k = key_of(v);
        if (k < in.key) continue;
        const int b1 = bin1(v);
        int bin = b1;
        if (level > 0) {
          if (b1 != want || k > khi || k < klo) continue;
          bin = (int)((khi - k) >> shift);
        }
        atomicAdd(&s.count[bin], 1u);
        if (mass) {
          const unsigned long long w = weight_of(v, sc, s.pow2);
          if (w) {
            const unsigned wl = (unsigned)w, old = atomicAdd(&s.lo[bin], wl);
            const unsigned wh = (unsigned)(w >> 32) + (old + wl < old ? 1u : 0u);
            if (wh) atomicAdd(&s.hi[bin], wh);
          }
        }
      }
      cluster_sync();
      // every CTA sums every bin over the cluster
      for (int i = tid; i < kSpBins; i += kSpThreads) {
        unsigned long long t = 0;
        for (uint32_t c = 0; c < ctas; ++c) {
          if (mass)
            t += ld_cluster_u32(cluster_addr(&s.lo[i], c)) + ((unsigned long long)ld_cluster_u32(cluster_addr(&s.hi[i], c)) << 32);
          else
            t += ld_cluster_u32(cluster_addr(&s.count[i], c));
        }
        s.sum[i] = t;
      }
      if (tid == 0) {
        s.found_bin = -1;
        s.found_above = 0;
      }
      __syncthreads();
      if (warp == 0) {
        // the first bin at which the running sum reaches the target
        unsigned long long run = above;
        for (int i0 = 0; i0 < kSpBins; i0 += 32) {
          unsigned long long v = s.sum[i0 + lane], inc = v;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, run + inc >= target);
          if (hit) {
            const int f = __ffs(hit) - 1;
            if (lane == f) {
              s.found_bin = i0 + f;
              s.found_above = run + inc - v;
            }
            break;
          }
          run += __shfl_sync(0xffffffffu, inc, 31);
        }
      }
      cluster_sync();  // the histograms may be cleared again
      const int bin = s.found_bin;
      if (bin < 0) return out;  // (only at the first level, where the run is everything)
      above = s.found_above;
      if (level > 0 && shift == 0) {
        // a single value: as many of its equals as the target takes
        out.key = khi - (unsigned)bin;
        if (mass) {
          const unsigned long long w = weight_of(key_float(out.key), sc, s.pow2);
          out.ties = (target - above + w - 1) / w;
        } else {
          out.ties = target - above;
        }
        return out;
      }
      if (level == 0) {
        want = bin;
        // the keys of the bin's values: their bounds over the cluster
        unsigned lo = 0xffffffffu, hi = 0u;
        for (int i = tid; i < n; i += kSpThreads) {
          const float v = value_at(a, held, src, base, i);
          if (!(v >= -FLT_MAX) || bin1(v) != want) continue;
          const unsigned k = key_of(v);
          if (k < in.key) continue;
          lo = min(lo, k);
          hi = max(hi, k);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        __syncthreads();
        if (lane == 0) {
          s.warp_a[warp] = lo;
          s.warp_b[warp] = hi;
        }
        __syncthreads();
        for (int w = 0; w < kSpWarps; ++w) {
          lo = min(lo, (unsigned)s.warp_a[w]);
          hi = max(hi, (unsigned)s.warp_b[w]);
        }
        exchange(s, 1, lo, hi, rank, ctas);
        klo = 0xffffffffu;
        khi = 0;
        for (uint32_t c = 0; c < ctas; ++c) {
          klo = min(klo, (unsigned)s.board[1].a[c]);
          khi = max(khi, (unsigned)s.board[1].b[c]);
        }
      } else {
        const unsigned top = khi - ((unsigned)bin << shift);
        const unsigned span = (1u << shift) - 1;
        klo = top - klo < span ? klo : top - span;
        khi = top;
      }
      shift = 0;
      while (((khi - klo) >> shift) >= kSpBins) ++shift;
    }
  };

  // The kept mass and count of this slice under the cut and min_p's floor.
  auto kept_of = [&](unsigned long long& mass, unsigned long long& count) {
    mass = count = 0;
    // ties in the slices before this one
    unsigned long long eq = 0, none = 0;
    if (cut.key && cut.ties != ~0ull) {
      for (int i = tid; i < n; i += kSpThreads) {
        const float v = value_at(a, held, src, base, i);
        eq += v >= -FLT_MAX && key_of(v) == cut.key;
      }
      cta_sum(s, eq, none);
      exchange(s, 2, eq, 0, rank, ctas);
      ties_before = 0;
      for (uint32_t c = 0; c < rank; ++c) ties_before += s.board[2].a[c];
      const unsigned long long left = cut.ties > ties_before ? cut.ties - ties_before : 0;
      const unsigned long long in = min(left, eq);
      if (cut.key >= floor_key && tid == 0) {
        const unsigned long long w = greedy ? 1ull : weight_of(key_float(cut.key), sc, s.pow2);
        mass = in * w;
        count = in;
      }
    }
    const bool tied = cut.key && cut.ties != ~0ull;
    for (int i = tid; i < n; i += kSpThreads) {
      const float v = value_at(a, held, src, base, i);
      if (!(v >= -FLT_MAX)) continue;
      const unsigned k = key_of(v);
      if (k < floor_key || k < cut.key || (tied && k == cut.key)) continue;
      ++count;
      mass += greedy ? 1ull : weight_of(v, sc, s.pow2);
    }
    cta_sum(s, mass, count);
  };

  if (!bad && !greedy) {
    if (top_k > 0 && (unsigned long long)top_k < finite) cut = find_cut(false, (unsigned long long)top_k, cut);
    if (top_p < 1.f) {
      // the mass that top-k leaves
      const unsigned fk = floor_key;
      floor_key = 1u;
      unsigned long long mass, count;
      kept_of(mass, count);
      exchange(s, 3, mass, count, rank, ctas);
      unsigned long long all = 0;
      for (uint32_t c = 0; c < ctas; ++c) all += s.board[3].a[c];
      const unsigned long long f = fraction(top_p);
      const unsigned long long target = max(1ull, __umul64hi(all, f) + (all * f != 0 ? 1 : 0));
      const SpCut p = find_cut(true, target, cut);
      if (p.key > cut.key || (p.key == cut.key && p.ties < cut.ties)) cut = p;
      floor_key = fk;
    }
  }
  unsigned long long mass = 0, count = 0;
  if (!bad) kept_of(mass, count);
  cluster_sync();  // boards 3 and 0 were read
  exchange(s, 0, mass, count, rank, ctas);
  unsigned long long before = 0, mine = 0;
  kept = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    const unsigned long long x = s.board[0].a[c];
    if (c < rank) before += x;
    if (c == rank) mine = x;
    total += x;
    kept += s.board[0].b[c];
  }
  const unsigned long long target = __umul64hi(total, fraction(u));  // the first running sum above it
  if (bad) {
    if (rank == 0 && tid == 0) {
      a.token[row] = -1;
      if (a.logprob) a.logprob[row] = __uint_as_float(0x7fc00000u);
      if (a.kept) a.kept[row] = 0;
    }
    return;
  }
  if (target < before || target >= before + mine) return;  // drawn from another slice
  // ---- the token: the slice's running sum in index order, chunk by chunk
  unsigned long long run = before, seen = ties_before;
  const bool tied = cut.key && cut.ties != ~0ull;
  for (int i0 = 0; i0 < n; i0 += kSpThreads) {
    const int i = i0 + tid;
    const float v = i < n ? value_at(a, held, src, base, i) : __uint_as_float(0xff800000u);
    const bool fine = v >= -FLT_MAX;
    const unsigned k = key_of(v);
    const bool eq = fine && tied && k == cut.key;
    // places among the equal ones
    const unsigned be = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) s.warp_b[warp] = __popc(be);
    __syncthreads();
    unsigned long long place = seen + __popc(be & ((1u << lane) - 1));
    for (int w = 0; w < kSpWarps; ++w) {
      if (w < warp) place += s.warp_b[w];
      seen += s.warp_b[w];
    }
    const bool in = fine && k >= floor_key && (eq ? place < cut.ties : k >= cut.key);
    const unsigned long long w = in ? (greedy ? 1ull : weight_of(v, sc, s.pow2)) : 0ull;
    unsigned long long inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) s.warp_a[warp] = inc;
    __syncthreads();
    unsigned long long pre = run;
    for (int w2 = 0; w2 < kSpWarps; ++w2) {
      if (w2 < warp) pre += s.warp_a[w2];
      run += s.warp_a[w2];
    }
    if (in && pre + inc > target && pre + inc - w <= target) {
      a.token[row] = base + i;
      if (a.kept) a.kept[row] = (int)min(kept, (unsigned long long)INT_MAX);
      if (a.logprob)
        a.logprob[row] = greedy ? 0.f : (float)(((double)v - (double)sc.base) / (double)T -
                                                log((double)total) + 0.69314718055994530942 * (kSpTop - sc.nref));
    }
    if (run > target) break;
  }
}

// CTAs of a row's cluster: slices of some 4096 to 32768 values.
int sample_ctas(int V) { return V <= 4096 ? 1 : V <= 16384 ? 2 : V <= 32768 ? 4 : 8; }

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" dg_status dg_sample(const void* logits, int32_t bf16, int64_t ld, int32_t R, int32_t V, const dg_sampling* how,
                               const float* u, int32_t* token, float* logprob, int32_t* kept, void* stream) {
  if (!logits || !how || !u || !token || R <= 0 || V <= 0 || (R > 1 && ld < V)) return DG_ERR_ARG;
  const uintptr_t words = reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(token) |
                          reinterpret_cast<uintptr_t>(logprob) | reinterpret_cast<uintptr_t>(kept) |
                          reinterpret_cast<uintptr_t>(how->temperature) | reinterpret_cast<uintptr_t>(how->top_p) |
                          reinterpret_cast<uintptr_t>(how->min_p) | reinterpret_cast<uintptr_t>(how->top_k);
  if (words % 4 || reinterpret_cast<uintptr_t>(logits) % (bf16 ? 2 : 4)) return DG_ERR_ARG;
  if (V > kSpMaxV) return DG_ERR_SHAPE;
  static const SpTables tables = [] {
    SpTables t;
    for (int j = 0; j < kSpTable; ++j) t.t[j] = (uint32_t)std::llround(std::ldexp(std::exp2(j / 64.0), 29));
    return t;
  }();
  const int ctas = sample_ctas(V);
  SpArgs a{};
  a.logits = logits;
  a.u = u;
  a.temperature = how->temperature;
  a.top_p = how->top_p;
  a.min_p = how->min_p;
  a.top_k = how->top_k;
  a.token = token;
  a.kept = kept;
  a.logprob = logprob;
  a.ld = ld;
  a.R = R;
  a.V = V;
  a.slice = cdiv(cdiv(V, ctas), 8) * 8;
  a.held = a.slice < kSpHeld ? a.slice : kSpHeld;
  a.bf16 = bf16 != 0;
  a.temperature_all = how->temperature_all;
  a.top_p_all = how->top_p_all;
  a.min_p_all = how->min_p_all;
  a.top_k_all = how->top_k_all;
  cudaError_t e = set_smem_once<sample_kernel>(kSpHeld * (int)sizeof(float));
  if (e != cudaSuccess) return DG_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(R, ctas);
  cfg.blockDim = dim3(kSpThreads);
  cfg.dynamicSmemBytes = sizeof(float) * a.held;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = ctas;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = kProgrammaticLaunch;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, sample_kernel, a, tables);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

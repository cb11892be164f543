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
// the weights' own 2^-28.
//
// A cluster of CTAs takes a row: each holds a slice in shared memory, read once from
// global memory (what bounds the call), and the passes over it are on chip.  A cut is
// searched in three steps:
//   a sample of the slices, in a histogram linear in the value below the maximum, gives
//     a bracket of values in which the border most likely lies
//   one pass over all values: what lies above the bracket is summed in registers, what
//     lies in it goes into 2048 bins of a second histogram (atomics for a few per cent
//     of the values; all of them through atomics took three times as long)
//   the values of the bin that holds the border, a few, are compared with one another
// Where the border is not in the bracket, or too many different values share its bin,
// histograms of all values, refined over the bits of the values, find it instead.
#include <cfloat>
#include <climits>
#include <atomic>
#include <cmath>

#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kSpThreads = 512;
constexpr int kSpWarps = kSpThreads / 32;
constexpr int kSpBins = 2048;
constexpr int kSpMaxV = 1 << 20;
constexpr int kSpList = 512;                  // keys of a bin that are compared with one another
constexpr int kSpSide = 512;                  // sampled values on either side of a bracket
constexpr int kSpMaxCluster = 16;
constexpr int kSpTable = 128;                 // 2^(j / 128)
constexpr int kSpTop = 43;                    // a weight of the row's scale is 2^43: 2^20 of them stay below 2^63
constexpr float kSpUnit = 32.0f;              // bins of the first histogram to a factor of two in weight
constexpr int kSpSample = 16384;              // longer vocabularies are sampled first
constexpr int kSpHeld = 43008;                // most values of a slice held in shared memory

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
  uint32_t t[kSpTable];  // 2^29 2^(j / 128), rounded
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
  unsigned long long sum[kSpBins];        // the bins, summed over the cluster; then the cluster's list, below
  uint2 pow2[kSpTable];                   // the table entry as an integer and as a float
  SpBoard board[5];
  unsigned long long warp_a[kSpWarps], warp_b[kSpWarps];
  unsigned list[kSpList];                 // this CTA's keys in the border's bin
  unsigned long long found_total;
  unsigned listed;
  unsigned long long found_above;
  int found_bin;
  unsigned cut_key;
  unsigned long long cut_ties;
  float bracket_hi, bracket_lo;
  SpScale scale;
  unsigned floor_key;
};

DG_DEV unsigned ld_cluster_u32(uint32_t a) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
DG_DEV void st_cluster_u32(uint32_t a, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
DG_DEV void st_cluster_u64(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// The weight of a value, 2^(x - nref + 43) rounded down to a whole number.  x = l c is
// taken as a sum of two floats, so that r = x - k / 128 keeps all its bits; 2^(k / 128)
// comes from the table and 2^r - 1 from three terms of its series (the fourth is
// below 2^-38); their product is added in units of 2^-29 of the table's scale.
DG_DEV unsigned long long weight_of(float v, const SpScale& s, const uint2* pow2) {
  const float l = v - s.base;
  const float x = l * s.c;
  float e = fmaf(l, s.c, -x);
  e = fmaf(l, s.clo, e);
  // values far below the largest weigh nothing (and x may be -inf)
  if (!(x > (float)(s.nref - 64))) return 0ull;
  // 128 x, rounded: the sum with 1.5 2^23 holds it in its low bits (|x| is below 2^15)
  const float y = fmaf(x, 128.0f, 12582912.0f);
  const int k = __float_as_int(y) - 0x4b400000;
  const float r = fmaf(y - 12582912.0f, -0.0078125f, x) + e;
  const float q = r * fmaf(r, fmaf(r, 0.05550410866f, 0.2402265070f), 0.6931471806f);
  const uint2 t = pow2[k & (kSpTable - 1)];
  // t q, rounded, the same way (below 2^22)
  const unsigned m = t.x + (__float_as_uint(fmaf(__uint_as_float(t.y), q, 12582912.0f)) - 0x4b400000u);
  return ((unsigned long long)m << 32) >> min(32 + 29 - kSpTop + s.nref - (k >> 7), 63);  // by 19 and more
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

// The order of values; -0 and 0 are equal.
DG_DEV unsigned key_of(float v) { return float_key(v == 0.f ? 0.f : v); }

// The cut of a leading run: values above `key` are in, and of those equal to it the
// first `ties` by index.
struct SpCut {
  unsigned key;
  unsigned long long ties;
};

__global__ void __launch_bounds__(kSpThreads, 2) sample_kernel(SpArgs a, SpTables tables) {
  extern __shared__ __align__(16) float held[];
  __shared__ SpShared s;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t ctas = gridDim.y, rank = cluster_ctarank();
  const int row = blockIdx.x;
  const char* src = static_cast<const char*>(a.logits) + (size_t)row * a.ld * (a.bf16 ? 2 : 4);
  const int base = (int)rank * a.slice;
  const int n = max(0, min(a.slice, a.V - base));  // this CTA's values
  const int n4 = (n + 3) / 4;
  pdl_wait();
  for (int i = tid; i < kSpTable; i += kSpThreads) s.pow2[i] = make_uint2(tables.t[i], __float_as_uint((float)tables.t[i]));

  const float T = a.temperature ? a.temperature[row] : a.temperature_all;
  const float top_p = a.top_p ? a.top_p[row] : a.top_p_all, min_p = a.min_p ? a.min_p[row] : a.min_p_all;
  const int top_k = a.top_k ? a.top_k[row] : a.top_k_all;
  const float u = a.u[row];
  bool bad = !(T >= 0.f && T <= FLT_MAX) || !(top_p >= 0.f) || !(min_p >= 0.f && min_p <= 1.f) || top_k < 0 || !(u >= 0.f && u < 1.f);

  const float kNone = __uint_as_float(0xff800000u);  // -inf: behind the end, or banned
  auto load1 = [&](int i) {
    if (i >= n) return kNone;
    return a.bf16 ? __uint_as_float((unsigned)reinterpret_cast<const uint16_t*>(src)[base + i] << 16)
                  : __ldcs(reinterpret_cast<const float*>(src) + base + i);
  };
  // four values from i = 4 j on, from global memory
  const bool vec = (reinterpret_cast<uintptr_t>(src) + (size_t)base * (a.bf16 ? 2 : 4)) % (a.bf16 ? 8 : 16) == 0;
  auto load4 = [&](int j) {
    if (vec && 4 * j + 4 <= n) {
      if (!a.bf16) return __ldcs(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(src) + base) + j);
      const uint2 w = __ldcs(reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(src) + base) + j);
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xffff0000u));
    }
    return make_float4(load1(4 * j), load1(4 * j + 1), load1(4 * j + 2), load1(4 * j + 3));
  };
  const int held4 = a.held / 4;
  auto value4 = [&](int j) { return j < held4 ? reinterpret_cast<const float4*>(held)[j] : load4(j); };

  // ---- the slice, its largest value, its finite ones
  float top = kNone, low = __uint_as_float(0x7f800000u);
  bool fine = true;
  unsigned fin = 0;
#pragma unroll 4
  for (int j = tid; j < n4; j += kSpThreads) {
    const float4 v = load4(j);
    if (j < held4) reinterpret_cast<float4*>(held)[j] = v;
    const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      top = fmaxf(top, w[e]);
      if (w[e] >= -FLT_MAX) low = fminf(low, w[e]);
      fine = fine && w[e] <= FLT_MAX;
      fin += w[e] >= -FLT_MAX;
    }
  }
  unsigned mkey = __reduce_max_sync(0xffffffffu, top >= -FLT_MAX ? key_of(top) : 0u);
  const unsigned wrong = __any_sync(0xffffffffu, !fine) ? 1u : 0u;
  fin = __reduce_add_sync(0xffffffffu, fin);
  unsigned lowest = __reduce_min_sync(0xffffffffu, low <= FLT_MAX ? key_of(low) : 0xffffffffu);
  if (lane == 0) {
    s.warp_a[warp] = ((unsigned long long)wrong << 32) | mkey;
    s.warp_b[warp] = ((unsigned long long)lowest << 32) | fin;
  }
  cluster_sync();  // (every CTA of the cluster runs before another writes to it)
  unsigned long long mw = 0, fin_here = 0;
  for (int w = 0; w < kSpWarps; ++w) {
    const unsigned long long x = s.warp_a[w];
    mw = ((mw | x) >> 32 << 32) | max((unsigned)mw, (unsigned)x);
    fin_here += (unsigned)s.warp_b[w];
    lowest = min(lowest, (unsigned)(s.warp_b[w] >> 32));
  }
  exchange(s, 0, mw, ((unsigned long long)lowest << 32) | fin_here, rank, ctas);
  unsigned long long finite = 0;
  mkey = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    mkey = max(mkey, (unsigned)s.board[0].a[c]);
    bad |= (s.board[0].a[c] >> 32) != 0;
    finite += (unsigned)s.board[0].b[c];
    lowest = min(lowest, (unsigned)(s.board[0].b[c] >> 32));
  }
  bad |= finite == 0;
  if (bad) {
    if (rank == 0 && tid == 0) {
      a.token[row] = -1;
      if (a.logprob) a.logprob[row] = __uint_as_float(0x7fc00000u);
      if (a.kept) a.kept[row] = 0;
    }
    return;
  }
  const float m = key_float(mkey);

  // Everything from here on is the same in all CTAs of the cluster but for their
  // slices, so that they come to every exchange together.
  SpCut cut{0u, ~0ull};       // all
  const bool greedy = T < 5.421010862427522e-20f || top_k == 1;  // 2^-64
  if (tid == 0) {  // in 64 bits, which few units compute
    unsigned fk = 1u;
    if (!greedy) {
      const double c = 1.4426950408889634074 / (double)T, xm = (double)m * c;
      const float base_v = fabs(xm) > 16384.0 ? m : 0.f;
      s.scale = SpScale{(float)c, (float)(c - (double)(float)c), base_v, (int)ceil(base_v != 0.f ? 0.0 : xm) + 1};
      if (min_p > 0.f) {
        // w >= min_p where l >= max + T ln(min_p): the first float at or above that border
        const double border = (double)m + (double)T * log((double)min_p);
        if (border >= -(double)FLT_MAX) {
          const float f = (float)border;
          fk = min(key_of(f) + ((double)f < border ? 1u : 0u), mkey);
        }
      }
    } else {
      s.scale = SpScale{0.f, 0.f, 0.f, 0};
    }
    s.floor_key = fk;
  }
  __syncthreads();
  const SpScale sc = s.scale;
  const unsigned floor_key = s.floor_key;  // min_p's: values at least this
  auto weight = [&](float v) { return greedy ? 1ull : weight_of(v, sc, s.pow2); };

  // ------------------------------------------------ histograms over the cluster
  auto clear = [&](bool mass) {
    for (int i = tid; i < kSpBins; i += kSpThreads) {
      s.count[i] = 0u;
      if (mass) s.lo[i] = s.hi[i] = 0u;
    }
    if (tid == 0) {
      s.found_bin = -1;
      s.found_above = 0;
      s.listed = 0;
    }
    __syncthreads();
  };
  auto add_mass = [&](int bin, unsigned long long w) {
    if (!w) return;
    const unsigned wl = (unsigned)w, old = atomicAdd(&s.lo[bin], wl);
    const unsigned wh = (unsigned)(w >> 32) + (old + wl < old ? 1u : 0u);
    if (wh) atomicAdd(&s.hi[bin], wh);
  };
  // s.sum: the bins' masses (what = 1) or counts (0), or with what = 2 the counts above
  // the 32 bits of `lo`, over the cluster: each CTA adds up some bins and tells all.
  auto combine = [&](int what) {
    cluster_sync();
    const int per = kSpBins / (int)ctas, b0 = (int)rank * per;
    for (int i = b0 + tid; i < b0 + per; i += kSpThreads) {
      unsigned long long t = 0;
#pragma unroll 4
      for (uint32_t c = 0; c < ctas; ++c) {
        unsigned long long x;
        if (what == 0) x = ld_cluster_u32(cluster_addr(&s.count[i], c));
        else {
          x = ld_cluster_u32(cluster_addr(&s.lo[i], c));
          x += (unsigned long long)ld_cluster_u32(cluster_addr(what == 1 ? &s.hi[i] : &s.count[i], c)) << 32;
        }
        t += x;
      }
      for (uint32_t c = 0; c < ctas; ++c) st_cluster_u64(cluster_addr(&s.sum[i], c), t);
    }
    cluster_sync();
  };
  // The inclusive running sum at a thread's four bins 4 tid .. 4 tid + 3
  auto scan_bins = [&](unsigned long long (&run)[4], auto&& of) {
    unsigned long long t = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) run[e] = t += of(4 * tid + e);
    unsigned long long inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31) s.warp_a[warp] = inc;
    __syncthreads();
    unsigned long long before = inc - t;
    for (int w = 0; w < warp; ++w) before += s.warp_a[w];
#pragma unroll
    for (int e = 0; e < 4; ++e) run[e] += before;
    __syncthreads();
  };
  // The first bin at which above + the running sum reaches the target: s.found_bin, and
  // what lies above it, s.found_above.
  auto find_bin = [&](unsigned long long above, unsigned long long target) {
    unsigned long long run[4];
    scan_bins(run, [&](int i) { return s.sum[i]; });
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned long long v = s.sum[4 * tid + e];
      if (above + run[e] >= target && above + run[e] - v < target) {
        s.found_bin = 4 * tid + e;
        s.found_above = above + run[e] - v;
      }
    }
    if (tid == kSpThreads - 1) s.found_total = above + run[3];
    __syncthreads();
  };
  // bins of the first histogram: linear below the maximum
  auto bin1 = [&](float v) { return (int)fminf((m - v) * (sc.c * kSpUnit), (float)(kSpBins - 1)); };

  // One cut: the smallest leading run of the values above key `in` whose count or mass
  // reaches `target`; the run is there.  Histograms of all values, refined.
  auto find_slowly = [&](bool mass, unsigned long long target, unsigned in) {
    unsigned khi = mkey, klo = 0;
    int shift = -1, want = -1;         // first level: linear in the value
    unsigned long long above = 0;      // what lies above the bin under search
    SpCut out{0u, ~0ull};
    for (int level = 0; level < 6; ++level) {
      clear(mass);
      unsigned lo_key = 0xffffffffu, hi_key = 0u;
      for (int j = tid; j < n4; j += kSpThreads) {
        const float4 v4 = value4(j);
        const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = vs[e];
          if (!(v >= -FLT_MAX)) continue;
          const unsigned k = key_of(v);
          if (k <= in) continue;
          const int b1 = bin1(v);
          int bin = b1;
          if (level > 0) {
            if (b1 != want || k > khi || k < klo) continue;
            bin = (int)((khi - k) >> shift);
          }
          if (mass) add_mass(bin, weight(v));
          else atomicAdd(&s.count[bin], 1u);
        }
      }
      combine(mass ? 1 : 0);
      find_bin(above, target);
      const int bin = s.found_bin;
      above = s.found_above;
      if (bin < 0) return out;
      if (level > 0 && shift == 0) {
        // a single value: as many of its equals as the target takes
        const unsigned long long w = mass ? weight(key_float(khi - (unsigned)bin)) : 1ull;
        out.key = khi - (unsigned)bin;
        out.ties = w ? (target - above + w - 1) / w : 1;
        cluster_sync();
        return out;
      }
      if (level == 0) {
        want = bin;
        // the bounds of the bin's keys over the cluster
        for (int j = tid; j < n4; j += kSpThreads) {
          const float4 v4 = value4(j);
          const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = vs[e];
            const unsigned k = key_of(v);
            if (!(v >= -FLT_MAX) || k <= in || bin1(v) != want) continue;
            lo_key = min(lo_key, k);
            hi_key = max(hi_key, k);
          }
        }
        lo_key = __reduce_min_sync(0xffffffffu, lo_key);
        hi_key = __reduce_max_sync(0xffffffffu, hi_key);
        __syncthreads();
        if (lane == 0) {
          s.warp_a[warp] = lo_key;
          s.warp_b[warp] = hi_key;
        }
        __syncthreads();
        for (int w = 0; w < kSpWarps; ++w) {
          lo_key = min(lo_key, (unsigned)s.warp_a[w]);
          hi_key = max(hi_key, (unsigned)s.warp_b[w]);
        }
        exchange(s, 1, lo_key, hi_key, rank, ctas);
        klo = 0xffffffffu;
        khi = 0;
        for (uint32_t c = 0; c < ctas; ++c) {
          klo = min(klo, (unsigned)s.board[1].a[c]);
          khi = max(khi, (unsigned)s.board[1].b[c]);
        }
      } else {
        const unsigned t = khi - ((unsigned)bin << shift), span = (1u << shift) - 1;
        klo = t - klo < span ? klo : t - span;
        khi = t;
      }
      shift = 0;
      while (((khi - klo) >> shift) >= kSpBins) ++shift;
    }
    return out;
  };

  // A bracket of values around the border, from a sample of the slices: about kSpSide
  // sampled values on either side.  share: the border's share of the sample's mass, or
  // rank its place among all values.
  auto sample_bracket = [&](bool mass, float share, unsigned long long place) {
    clear(true);
    const int bits = 28 - (32 - __clz(a.slice / 8));  // so that the whole sample's sum fits 32
    for (int j = tid; j < n4; j += 2 * kSpThreads) {
      const float v = value4(j).x;  // every eighth value
      if (!(v >= -FLT_MAX)) continue;
      const int b = bin1(v);
      atomicAdd(&s.count[b], 1u);
      if (mass) atomicAdd(&s.lo[b], (unsigned)(weight(v) >> (kSpTop - bits)));
    }
    combine(2);
    unsigned long long run[4], count[4];
    scan_bins(run, [&](int i) { return s.sum[i] & 0xffffffffull; });
    scan_bins(count, [&](int i) { return s.sum[i] >> 32; });
    // the estimated bin: where the running mass (or eight times the count) reaches the border
    if (tid == kSpThreads - 1) s.warp_b[0] = run[3];
    if (tid == 0) {
      s.bracket_hi = m;
      s.bracket_lo = kNone;
      s.found_above = ~0ull;  // the estimated place in the sample
    }
    __syncthreads();
    const float goal = fmaxf(mass ? share * (float)s.warp_b[0] : (float)place * 0.125f, 1e-30f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned long long x = s.sum[4 * tid + e];
      const float now = mass ? (float)run[e] : (float)count[e];
      const float was = mass ? (float)(run[e] - (x & 0xffffffffull)) : (float)(count[e] - (x >> 32));
      if (was < goal && now >= goal) s.found_above = count[e];
    }
    __syncthreads();
    const unsigned long long at = s.found_above;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int b = 4 * tid + e;
      const unsigned long long prev = count[e] - (s.sum[b] >> 32);
      const float unit = 1.0f / (sc.c * kSpUnit);
      // the last bin that ends kSpSide before, the first that ends kSpSide behind
      if (at != ~0ull && count[e] + kSpSide <= at && b + 1 < kSpBins && count[e] + kSpSide + (s.sum[b + 1] >> 32) > at)
        s.bracket_hi = m - (float)(b + 1) * unit;
      if (at != ~0ull && count[e] >= at + kSpSide && prev < at + kSpSide && b < kSpBins - 1) s.bracket_lo = m - (float)(b + 1) * unit;
    }
    __syncthreads();
  };

  // the cluster's keys of the border's bin and their weights, where the sums were
  unsigned* list_all = reinterpret_cast<unsigned*>(s.sum);
  unsigned long long* list_weight = s.sum + kSpList / 2;

  // What is kept of this slice, where a search has added it up already
  bool saved = false;
  unsigned long long mass_here = 0, count_here = 0, equal_here = 0;

  // One cut, by a bracket [lo, hi] of values: the smallest leading run of the values
  // above key `in` (0: all) whose count, or mass with p times their sum (and `more`, the
  // weight of values equal to `in` that count too), reaches the target.  floored: what
  // lies below the bracket is of no matter.
  auto find_cut = [&](bool mass, unsigned long long target, unsigned long long p, unsigned in, unsigned long long more, float lo,
                      float hi, bool floored, SpCut& out) {
    const float scale = fminf((float)(kSpBins - 1) / (hi - lo), FLT_MAX);
    auto bin2 = [&](float v) { return (int)fminf((hi - v) * scale, (float)(kSpBins - 1)); };
    clear(mass);
    unsigned long long above = 0, all = 0;
    unsigned nabove = 0;
    auto put = [&](float v) {
      if (!(v >= lo)) return;
      const unsigned k = key_of(v);
      if (k <= in) return;
      if (v > hi) {
        ++nabove;
        return;
      }
      atomicAdd(&s.count[bin2(v)], 1u);
    };
    auto put_mass = [&](float v) {
      if (in && key_of(v) <= in) return;
      const unsigned long long w = weight(v);
      all += w;
      if (v > hi) {
        above += w;
        ++nabove;
      } else if (v >= lo) {
        const int b = bin2(v);
        atomicAdd(&s.count[b], 1u);
        add_mass(b, w);
      }
    };
    if (mass) {
      const bool few = in != 0;
      const float least = few ? key_float(in) : kNone;
      for (int j = tid; j < n4; j += kSpThreads) {
        const float4 v = value4(j);
        if (few && fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) < least) continue;
        put_mass(v.x);
        put_mass(v.y);
        put_mass(v.z);
        put_mass(v.w);
      }
    } else {
      for (int j = tid; j < n4; j += kSpThreads) {
        const float4 v = value4(j);
        if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) < lo) continue;
        put(v.x);
        put(v.y);
        put(v.z);
        put(v.w);
      }
    }
    unsigned long long na = nabove, none = 0;
    cta_sum(s, above, all);
    cta_sum(s, na, none);
    const unsigned long long above_here = mass ? above : na;
    // the masses of the bins (or their counts), what lies above, the sum of all
    if (tid < ctas) {
      st_cluster_u64(cluster_addr(&s.board[2].a[rank], tid), above_here);
      st_cluster_u64(cluster_addr(&s.board[2].b[rank], tid), all);
    }
    combine(mass ? 1 : 0);
    above = all = 0;
    for (uint32_t c = 0; c < ctas; ++c) {
      above += s.board[2].a[c];
      all += s.board[2].b[c];
    }
    if (mass) {
      all += more;
      target = max(1ull, __umul64hi(all, p) + (all * p != 0 ? 1 : 0));
    }
    find_bin(above, target);
    const int bin = s.found_bin;
    if (bin < 0) {
      const unsigned long long t = s.found_total;
      if (t < target && in) {
        // within the values equal to `in`, which are not in the histogram
        const unsigned long long w = weight(key_float(in));
        out.key = in;
        out.ties = w ? (target - t + w - 1) / w : 1;
        return;
      }
      if (t < target && floored) return;  // min_p's floor cuts first
      out = find_slowly(mass, target, in);
      return;
    }
    const unsigned long long before = s.found_above;
    // the bin's keys: their bounds, their number, and as many as fit in the list
    unsigned lo_key = 0xffffffffu, hi_key = 0u;
    for (int j = tid; j < n4; j += kSpThreads) {
      const float4 v4 = value4(j);
      if (fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w)) < lo) continue;
      const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = vs[e];
        if (!(v >= lo) || v > hi || bin2(v) != bin) continue;
        const unsigned k = key_of(v);
        if (k <= in) continue;
        lo_key = min(lo_key, k);
        hi_key = max(hi_key, k);
        const unsigned at = atomicAdd(&s.listed, 1u);
        if (at < kSpList) s.list[at] = k;
      }
    }
    lo_key = __reduce_min_sync(0xffffffffu, lo_key);
    hi_key = __reduce_max_sync(0xffffffffu, hi_key);
    __syncthreads();
    if (lane == 0) {
      s.warp_a[warp] = lo_key;
      s.warp_b[warp] = hi_key;
    }
    __syncthreads();
    for (int w = 0; w < kSpWarps; ++w) {
      lo_key = min(lo_key, (unsigned)s.warp_a[w]);
      hi_key = max(hi_key, (unsigned)s.warp_b[w]);
    }
    const unsigned here = s.listed;
    exchange(s, 3, ((unsigned long long)hi_key << 32) | lo_key, here, rank, ctas);
    lo_key = 0xffffffffu;
    hi_key = 0;
    unsigned first = 0, number = 0;
    for (uint32_t c = 0; c < ctas; ++c) {
      lo_key = min(lo_key, (unsigned)s.board[3].a[c]);
      hi_key = max(hi_key, (unsigned)(s.board[3].a[c] >> 32));
      if (c < rank) first += (unsigned)s.board[3].b[c];
      number += (unsigned)s.board[3].b[c];
    }
    if (lo_key != hi_key && number > kSpList) {
      out = find_slowly(mass, target, in);
      return;
    }
    if (lo_key == hi_key) {
      const unsigned long long w = mass ? weight(key_float(lo_key)) : 1ull;
      out.key = lo_key;
      out.ties = (target - before + w - 1) / w;
      cluster_sync();  // (the boards and lists are free again)
    } else {
      for (unsigned i = tid; i < here; i += kSpThreads)
        for (uint32_t c = 0; c < ctas; ++c) st_cluster_u32(cluster_addr(&list_all[first + i], c), s.list[i]);
      cluster_sync();
      if (tid < number) list_weight[tid] = mass ? weight(key_float(list_all[tid])) : 1ull;
      __syncthreads();
      if (tid < number) {
        const unsigned k = list_all[tid];
        unsigned long long over = before, same = 0;
        for (unsigned i = 0; i < number; ++i) {
          const unsigned o = list_all[i];
          if (o > k) over += list_weight[i];
          same += o == k;
        }
        if (over < target && over + same * list_weight[tid] >= target) {  // (every equal one says the same)
          s.cut_key = k;
          s.cut_ties = (target - over + list_weight[tid] - 1) / list_weight[tid];
        }
      }
      __syncthreads();
      out.key = s.cut_key;
      out.ties = s.cut_ties;
    }
    if (mass && !in) {
      // this slice's kept mass: above the bracket, in the bins before, and of the list
      unsigned long long w = 0, c = 0;
      for (int i = tid; i < bin; i += kSpThreads) {
        w += s.lo[i] + ((unsigned long long)s.hi[i] << 32);
        c += s.count[i];
      }
      unsigned long long eq = 0, zero = 0;
      if (lo_key == hi_key) {
        if (tid == 0) eq = here;
      } else {
        for (unsigned i = tid; i < here; i += kSpThreads) {
          if (s.list[i] > out.key) {
            w += weight(key_float(s.list[i]));
            ++c;
          }
          eq += s.list[i] == out.key;
        }
      }
      cta_sum(s, w, c);
      cta_sum(s, eq, zero);
      mass_here = above_here + w;
      count_here = na + c;
      equal_here = eq;
      saved = true;
    }
  };

  if (greedy) {
    cut.key = mkey;
    cut.ties = 1;
  } else {
    // without a bracket: down to the lowest value, or to where nothing weighs
    const float lowest_v = fmaxf(key_float(lowest), m - (float)kSpBins / (sc.c * kSpUnit));
    if (top_k > 0 && (unsigned long long)top_k < finite) {
      float lo = lowest_v, hi = m;
      if (a.V > kSpSample) {
        sample_bracket(false, 0.f, (unsigned long long)top_k);
        lo = fmaxf(lo, s.bracket_lo);
        hi = s.bracket_hi;
      }
      find_cut(false, (unsigned long long)top_k, 0, 0u, 0, lo, hi, false, cut);
    }
    if (top_p < 1.f) {
      const unsigned long long p = fraction(top_p);
      SpCut c{0u, ~0ull};
      if (cut.key) {
        const unsigned long long w = weight(key_float(cut.key));
        find_cut(true, 0, p, cut.key, cut.ties * w, key_float(cut.key), m, false, c);
      } else {
        float lo = lowest_v, hi = m;
        if (floor_key > 1u) lo = key_float(floor_key);  // what lies below is not kept anyway
        else if (a.V > kSpSample) {
          sample_bracket(true, top_p, 0);
          lo = fmaxf(lo, s.bracket_lo);
          hi = s.bracket_hi;
        }
        find_cut(true, 0, p, 0u, 0, lo, hi, floor_key > 1u, c);
      }
      if (c.key) cut = c;
    }
  }
  // min_p's floor, where it is tighter
  const bool tied = cut.key && cut.ties != ~0ull && cut.key >= floor_key;
  const unsigned least = max(cut.key, floor_key);  // above it (tied), or from it on
  auto in_run = [&](unsigned k) { return tied ? k > cut.key : k >= least; };
  const float least_v = key_float(max(least, 0x00800000u));  // no finite value is below

  // ---- this slice's kept mass and count
  if (!(saved && tied)) {
    unsigned long long w = 0, c = 0, eq = 0, zero = 0;
    for (int j = tid; j < n4; j += kSpThreads) {
      const float4 v4 = value4(j);
      if (!(fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w)) >= least_v)) continue;
      const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = vs[e];
        if (!(v >= -FLT_MAX)) continue;
        const unsigned k = key_of(v);
        if (in_run(k)) {
          ++c;
          w += weight(v);
        }
        eq += tied && k == cut.key;
      }
    }
    cta_sum(s, w, c);
    cta_sum(s, eq, zero);
    mass_here = w;
    count_here = c;
    equal_here = eq;
  }
  const unsigned long long w_tie = tied ? weight(key_float(cut.key)) : 0ull;
  // equal ones are taken in the order of the slices
  if (tid < ctas) st_cluster_u64(cluster_addr(&s.board[4].a[rank], tid), mass_here);
  if (tid < ctas) st_cluster_u64(cluster_addr(&s.board[4].b[rank], tid), (count_here << 32) | equal_here);
  cluster_sync();
  unsigned long long total = 0, kept = 0, before = 0, mine = 0, left = tied ? cut.ties : 0, left_here = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    const unsigned long long eq = s.board[4].b[c] & 0xffffffffull, take = min(left, eq);
    const unsigned long long x = s.board[4].a[c] + take * w_tie;
    if (c < rank) before += x;
    if (c == rank) {
      mine = x;
      left_here = take;
    }
    left -= take;
    total += x;
    kept += (s.board[4].b[c] >> 32) + take;
  }
  const unsigned long long target = __umul64hi(total, fraction(u));  // the first running sum above it
  if (target < before || target >= before + mine) return;  // drawn from another slice

  // ---- the token: a warp takes a run of the slice; the run that holds the border is
  // gone through by its warp
  const int run4 = ((n4 + kSpWarps - 1) / kSpWarps + 31) / 32 * 32, j0 = warp * run4, j1 = min(n4, j0 + run4);
  unsigned long long w = 0, eq = 0;
  for (int j = j0 + lane; j < j1; j += 32) {
    const float4 v4 = value4(j);
    if (!(fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w)) >= least_v)) continue;
    const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = vs[e];
      if (!(v >= -FLT_MAX)) continue;
      const unsigned k = key_of(v);
      if (in_run(k)) w += weight(v);
      eq += tied && k == cut.key;
    }
  }
  w = warp_sum(w);
  eq = warp_sum(eq);
  __syncthreads();
  if (lane == 0) {
    s.warp_a[warp] = w;
    s.warp_b[warp] = eq;
  }
  __syncthreads();
  unsigned long long run = before;
  left = left_here;
  for (int x = 0; x < warp; ++x) {
    const unsigned long long take = min(left, s.warp_b[x]);
    run += s.warp_a[x] + take * w_tie;
    left -= take;
  }
  if (target < run || target >= run + s.warp_a[warp] + min(left, s.warp_b[warp]) * w_tie) return;
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    const float4 v4 = j < j1 ? value4(j) : make_float4(kNone, kNone, kNone, kNone);
    const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
    unsigned long long ws[4], sum = 0;
    unsigned equal = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned k = key_of(vs[e]);
      const bool there = vs[e] >= -FLT_MAX;
      ws[e] = there && in_run(k) ? weight(vs[e]) : 0ull;
      equal |= (there && tied && k == cut.key ? 1u : 0u) << e;
    }
    // the equal ones' places
    unsigned places = __popc(equal), upto = places;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    unsigned long long place = upto - places;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (equal >> e & 1) {
        if (place < left) ws[e] = w_tie;
        ++place;
      }
      sum += ws[e];
    }
    unsigned long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    unsigned long long now = run + inc - sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (ws[e] && target >= now && target < now + ws[e]) {
        const float v = vs[e];
        a.token[row] = base + 4 * j + e;
        if (a.kept) a.kept[row] = (int)min(kept, (unsigned long long)INT_MAX);
        if (a.logprob)
          a.logprob[row] = greedy ? 0.f : (float)(((double)v - (double)sc.base) / (double)T -
                                                  log((double)total) + 0.69314718055994530942 * (kSpTop - sc.nref));
      }
      now += ws[e];
    }
    const unsigned total_eq = __shfl_sync(0xffffffffu, upto, 31);
    left -= min(left, (unsigned long long)total_eq);
    run += __shfl_sync(0xffffffffu, inc, 31);
    if (run > target) return;
  }
}

// CTAs of a row's cluster: slices of up to 16384 values, so that two CTAs share an SM
// and one row's values come while another's are worked on.
int sample_ctas(int V) {
  int c = 1;
  while (c < kSpMaxCluster && (int64_t)c * 16384 < V) c *= 2;
  return c;
}

// Clusters of 16, once on each device.
cudaError_t allow_large_clusters() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(reinterpret_cast<const void*>(sample_kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

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
    for (int j = 0; j < kSpTable; ++j) t.t[j] = (uint32_t)std::llround(std::ldexp(std::exp2(j / (double)kSpTable), 29));
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
  if (e == cudaSuccess) e = allow_large_clusters();
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

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
// A cluster of CTAs takes a row, a slice each; a warp a run of its CTA's slice.  What
// bounds few rows is the chain of dependent steps (one row of 262144: 29 us, five
// exchanges of the cluster among them), many rows the instructions of an exact weight
// (some 50 a value; 256 rows of 262144: 263 us, 268 MB read once from HBM; for the rows
// under way they are read again from L2).  The passes:
//   the largest value
//   where a cut is asked for, a sample: its histogram, linear in the value below the
//     maximum, gives a bracket of values in which the border most likely lies
//   all values, with their weights: what lies above the bracket is summed in registers,
//     what lies in it (some thousand values) goes into lists in index order
// Then one CTA, the leader, has the lists and the runs' sums in its shared memory and
// finishes alone: it finds the border among the listed values, adds up what is kept of
// each run, and goes through the run in which the token lies.
// Where the border is not in the bracket, the exact sums say how far off the sample was
// and the pass is taken again; where that fails too, or too many values lie in the
// bracket, histograms of all values, refined over the bits of the values, find it.
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kSpThreads = 512;
constexpr int kSpWarps = kSpThreads / 32;
constexpr int kSpBins = 2048;
constexpr int kSpMaxV = 1 << 20;
constexpr int kSpKeys = 512;                  // keys of a bin that are compared with one another
constexpr int kSpSample = 8192;               // longer vocabularies are sampled first
constexpr int kSpSide = 384;                  // sampled values on either side of a bracket
constexpr int kSpTries = 3;
constexpr int kSpMaxCluster = 16;
constexpr int kSpRuns = kSpMaxCluster * kSpWarps;
constexpr int kSpCap = 640;                   // listed values of a run, over the CTAs of a row
constexpr int kSpSampled = 4;                 // sampled blocks of 128 values of a run, at most
constexpr int kSpTable = 128;                 // 2^(j / 128)
constexpr int kSpTop = 43;                    // a weight of the row's scale is 2^43: 2^20 of them stay below 2^63
constexpr float kSpFar = 64.0f;               // factors of two below the largest weight at which nothing weighs
constexpr float kNone = -INFINITY;            // behind the end, or banned

struct SpArgs {
  const void* logits;  // fp32 or bf16 [R][ld]
  const float *u, *temperature, *top_p, *min_p;
  const int* top_k;
  int32_t *token, *kept;
  float* logprob;
  int64_t ld;
  int R, V, slice, run4, step, bf16;  // step: a power of two
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

// The cut of a leading run: values above `key` are in, and of those equal to it the
// first `ties` by index.
struct SpCut {
  unsigned key;
  unsigned long long ties;
};

struct alignas(16) SpShared {
  unsigned count[kSpBins];
  unsigned lo[kSpBins], hi[kSpBins];      // masses, 64 bits in two words
  unsigned long long sum[kSpBins];        // the bins, summed over the cluster
  uint2 pow2[kSpTable];                   // the table entry as an integer and as a float
  SpBoard board[4];
  unsigned long long warp_a[kSpWarps], warp_b[kSpWarps], part[4][kSpWarps];
  // the leader's: of every run of the row, the mass and the number of values above the
  // bracket (or of all that is kept), how many are equal to the cut, how many listed
  unsigned long long run_mass[kSpRuns];
  unsigned run_count[kSpRuns], run_equal[kSpRuns], run_listed[kSpRuns];
  unsigned keys[kSpKeys];                 // the border's bin
  unsigned nkeys, key_lo, key_hi;
  unsigned long long found_above, found_total;
  int found_bin;
  SpCut cut;
  float bracket_hi, bracket_lo;
  SpScale scale;
  double ln_min_p;                        // T ln(min_p), worked out while the logits are on their way
  unsigned floor_key;
};

static_assert(sizeof(SpShared) % 16 == 0, "the lists lie behind it");
static_assert(kSpSampled * 128 <= kSpCap, "the samples lie where the lists will");
constexpr int kSpSmem = (int)sizeof(SpShared) + kSpWarps * kSpCap * 4;

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

// The weight of a value, 2^(x - nref + 43) rounded down to a whole number, as m << e.
// x = l c is taken as a sum of two floats, so that r = x - k / 128 keeps all its bits;
// 2^(k / 128) comes from the table and 2^r - 1 from three terms of its series (the
// fourth is below 2^-38); their product is added in units of 2^-29 of the table's scale.
struct SpWeight {
  unsigned m, p;  // m p
  DG_DEV void add_to(unsigned long long& sum) const { sum += (unsigned long long)m * p; }
};
DG_DEV SpWeight weight_parts(float v, const SpScale& s, const uint2* pow2) {
  const float l = v - s.base;
  const float x = l * s.c;
  float e = fmaf(l, s.c, -x);
  e = fmaf(l, s.clo, e);
  // 128 x, rounded: the sum with 1.5 2^23 holds it in its low bits (|x| is below 2^15)
  const float y = fmaf(x, 128.0f, 12582912.0f);
  const int k = __float_as_int(y) - 0x4b400000;
  const float r = fmaf(y - 12582912.0f, -0.0078125f, x) + e;
  const float q = r * fmaf(r, fmaf(r, 0.05550410866f, 0.2402265070f), 0.6931471806f);
  const uint2 t = pow2[k & (kSpTable - 1)];
  // t q, rounded, the same way (below 2^22)
  unsigned m = t.x + (__float_as_uint(fmaf(__uint_as_float(t.y), q, 12582912.0f)) - 0x4b400000u);
  // values far below the largest weigh nothing (and x may be -inf)
  if (!(x > (float)(s.nref - 64))) m = 0u;
  const int up = kSpTop - 29 - s.nref + (k >> 7), shift = min(max(up, 0), 31);
  return SpWeight{m >> min(shift - up, 31), 1u << shift};
}
DG_DEV unsigned long long weight_of(float v, const SpScale& s, const uint2* pow2) {
  const SpWeight w = weight_parts(v, s, pow2);
  return (unsigned long long)w.m * w.p;
}

// log2 of a sum of weights, to 2^-28: the table entry below its leading bits, and three
// terms of the series for the rest.  (A 64-bit log takes a microsecond here.)
DG_DEV double log2_of(unsigned long long sum, const uint2* pow2) {
  const int lead = __clzll(sum);
  const unsigned top = (unsigned)((sum << lead) >> 32);  // 2^31 times the mantissa
  const int j = min(kSpTable - 1, max(0, (int)(kSpTable * __log2f((float)top * 4.656612873077393e-10f))));
  const unsigned t = pow2[j].x << 2;
  const float r = (float)(int)(top - t) / (float)t;
  return (63 - lead) + j * (1.0 / kSpTable) + (double)(1.442695041f * (r * fmaf(r, fmaf(r, 0.333333333f, -0.5f), 1.0f)));
}

// ln(w / (w + rest)) for rest < w, to 2^-27 of itself: -2 atanh(z) with z = rest / (2 w +
// rest), which is 1/3 at most, in two floats, and nine terms of the series.
DG_DEV float ln_share(unsigned long long rest, unsigned long long w) {
  const double den = (double)(rest + 2 * w);
  const float z0 = (float)rest / (float)den, q = z0 * z0;
  const double z = (double)z0 + (double)((float)fma(-(double)z0, den, (double)rest) / (float)den);
  float t = 1.0f / 17;
#pragma unroll
  for (int n = 15; n >= 3; n -= 2) t = fmaf(t, q, 1.0f / n);
  return (float)(-2.0 * z * (1.0 + (double)(t * q)) + 0.0);
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

__global__ void __launch_bounds__(kSpThreads, 2) sample_kernel(SpArgs a, SpTables tables) {
  extern __shared__ __align__(16) char smem[];
  SpShared& s = *reinterpret_cast<SpShared*>(smem);
  // [run][cap] listed values, in any order: of the CTA's own runs, in the leader of all
  float* list_v = reinterpret_cast<float*>(smem + sizeof(SpShared));
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t ctas = gridDim.y, rank = cluster_ctarank();
  const int row = blockIdx.x;
  const int cap = kSpCap / (int)ctas, runs = (int)ctas * kSpWarps;
  const char* src = static_cast<const char*>(a.logits) + (size_t)row * a.ld * (a.bf16 ? 2 : 4);
  // every CTA of the cluster runs before another writes to it: waited for below
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  for (int i = tid; i < kSpTable; i += kSpThreads) s.pow2[i] = make_uint2(tables.t[i], __float_as_uint((float)tables.t[i]));

  const float T = a.temperature ? a.temperature[row] : a.temperature_all;
  const float top_p = a.top_p ? a.top_p[row] : a.top_p_all, min_p = a.min_p ? a.min_p[row] : a.min_p_all;
  const int top_k = a.top_k ? a.top_k[row] : a.top_k_all;
  const float u = a.u[row];
  bool bad = !(T >= 0.f && T <= FLT_MAX) || !(top_p >= 0.f) || !(min_p >= 0.f && min_p <= 1.f) || top_k < 0 || !(u >= 0.f && u < 1.f);

  if (tid == kSpThreads - 1 && min_p > 0.f) s.ln_min_p = (double)T * log((double)min_p);
  // four values from i on (a multiple of 4), -inf from `end` on
  const bool vec = reinterpret_cast<uintptr_t>(src) % (a.bf16 ? 8 : 16) == 0;
  auto load4 = [&](int i, int end) {
    if (vec && i + 4 <= end) {
      if (!a.bf16) return __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(src) + i));
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(src) + i));
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xffff0000u));
    }
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = i + e >= end ? kNone
             : a.bf16     ? __uint_as_float((unsigned)__ldg(reinterpret_cast<const uint16_t*>(src) + i + e) << 16)
                          : __ldg(reinterpret_cast<const float*>(src) + i + e);
    return make_float4(v[0], v[1], v[2], v[3]);
  };
  // f(four values, their place, the block of 128) for all of [i0, i1), a block of a warp at
  // a time (-inf behind the end, where the warp's other lanes still have some).  The loads
  // of whole blocks are D blocks ahead and ask nothing of their places.
  auto each4 = [&](auto depth, int i0, int i1, auto&& f) {
    constexpr int D = decltype(depth)::value;
    const int whole = vec ? (i1 - i0) >> 7 : 0, step = a.bf16 ? 256 : 512;
    const char* from = src + (size_t)(i0 + 4 * lane) * (a.bf16 ? 2 : 4);
    auto next = [&](int j) {
      const char* at = from + j * step;
      if (!a.bf16) return __ldg(reinterpret_cast<const float4*>(at));
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(at));
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xffff0000u));
    };
    float4 v[D];
#pragma unroll
    for (int j = 0; j < D; ++j)
      if (j < whole) v[j] = next(j);
    int i = i0 + 4 * lane, block = 0;
#pragma unroll 1
    while (block < whole) {
#pragma unroll
      for (int j = 0; j < D; ++j) {
        if (block >= whole) break;
        const float4 now = v[j];
        if (block + D < whole) v[j] = next(D);
        f(now, i, block);
        from += step;
        i += 128;
        ++block;
      }
    }
    // the last block's part, or all of a row that does not lie on 16 (8) bytes (loads ahead
    // of these gain nothing)
#pragma unroll 1
    for (; i - 4 * lane < i1; i += 128, ++block)
      f(i < i1 ? load4(i, i1) : make_float4(kNone, kNone, kNone, kNone), i, block);
  };
  using Ahead2 = std::integral_constant<int, 2>;
  using Ahead4 = std::integral_constant<int, 4>;
  // this warp's run: values [first, last)
  auto run_first = [&](int r) { return min(a.V, r / kSpWarps * a.slice + r % kSpWarps * a.run4 * 4); };
  auto run_last = [&](int r) { return min(min(a.V, (r / kSpWarps + 1) * a.slice), run_first(r) + a.run4 * 4); };
  const int mine = (int)rank * kSpWarps + warp, first = run_first(mine), last = run_last(mine);

  // ---- the largest value, the lowest, the number of finite ones
  float top = kNone, low = INFINITY;
  unsigned fin = 0;
  // every a.step-th 128 values are a run's sample, kept where its list will lie
  const bool sampled = a.V > kSpSample;
  const int step_log = 31 - __clz(a.step);
  float4* sample = reinterpret_cast<float4*>(list_v) + warp * kSpSampled * 32 + lane;
  each4(Ahead4{}, first, last, [&](const float4& v, int, int block) {
    if (sampled && (block & (a.step - 1)) == 0) sample[(block >> step_log) * 32] = v;
    // NaN goes through to the largest
    asm("max.NaN.f32 %0, %0, %1;\n max.NaN.f32 %0, %0, %2;\n max.NaN.f32 %0, %0, %3;\n max.NaN.f32 %0, %0, %4;"
        : "+f"(top)
        : "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w));
    const float least = fminf(fminf(v.x, v.y), fminf(v.z, v.w));
    if (least >= -FLT_MAX) {
      low = fminf(low, least);
      fin += 4;
    } else {
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const float x = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
        if (x >= -FLT_MAX) {
          low = fminf(low, x);
          ++fin;
        }
      }
    }
  });
  const bool fine = top <= FLT_MAX;
  unsigned mkey = __reduce_max_sync(0xffffffffu, top >= -FLT_MAX ? key_of(top) : 0u);
  unsigned lowest = __reduce_min_sync(0xffffffffu, low <= FLT_MAX ? key_of(low) : 0xffffffffu);
  const unsigned wrong = __any_sync(0xffffffffu, !fine) ? 1u : 0u;
  fin = __reduce_add_sync(0xffffffffu, fin);
  if (lane == 0) {
    s.warp_a[warp] = ((unsigned long long)wrong << 32) | mkey;
    s.warp_b[warp] = ((unsigned long long)lowest << 32) | fin;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  unsigned long long mw = 0, finite = 0;
  for (int w = 0; w < kSpWarps; ++w) {
    const unsigned long long x = s.warp_a[w];
    mw = ((mw | x) >> 32 << 32) | max((unsigned)mw, (unsigned)x);
    finite += (unsigned)s.warp_b[w];
    lowest = min(lowest, (unsigned)(s.warp_b[w] >> 32));
  }
  if (ctas > 1) {
    exchange(s, 0, mw, ((unsigned long long)lowest << 32) | finite, rank, ctas);
    finite = mw = 0;
    for (uint32_t c = 0; c < ctas; ++c) {
      const unsigned long long x = s.board[0].a[c];
      mw = ((mw | x) >> 32 << 32) | max((unsigned)mw, (unsigned)x);
      finite += (unsigned)s.board[0].b[c];
      lowest = min(lowest, (unsigned)(s.board[0].b[c] >> 32));
    }
  }
  mkey = (unsigned)mw;
  bad |= (mw >> 32) != 0 || finite == 0;
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
  // slices, so that they come to every exchange together, until the leader goes on alone.
  const bool greedy = T < 5.421010862427522e-20f || top_k == 1;  // 2^-64
  if (tid == 0) {
    unsigned fk = 1u;
    if (!greedy) {
      // log2(e) / T in two floats: the quotient, and what it leaves of log2(e) (exact) over T
      const float c = 1.44269502162933349609f / T, clo = (fmaf(-c, T, 1.44269502162933349609f) + 1.92596299112661e-8f) / T;
      const float base_v = fabsf(m * c) > 16384.0f ? m : 0.f;
      s.scale = SpScale{c, clo, base_v, base_v != 0.f ? 1 : (int)ceilf(m * c) + 1};
      if (min_p > 0.f) {
        // w >= min_p where l >= max + T ln(min_p): the first float at or above that border, worked out in 64 bits
        const double border = (double)m + s.ln_min_p;
        if (border >= -(double)FLT_MAX) {
          // (a key of a value: behind the negative value nearest to zero comes 0, not -0)
          const float f = (float)border;
          fk = min((double)f < border ? key_of(key_float(key_of(f) + 1u)) : key_of(f), mkey);
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

  // ---------------------------------------------------------------- histograms
  auto clear = [&](bool mass) {
    __syncthreads();  // what the last search left has been read by all
    for (int i = tid; i < kSpBins; i += kSpThreads) {
      s.count[i] = 0u;
      if (mass) s.lo[i] = s.hi[i] = 0u;
    }
    if (tid == 0) {
      s.found_bin = -1;
      s.found_above = 0;
      s.nkeys = 0;
      s.key_lo = 0xffffffffu;
      s.key_hi = 0;
    }
    __syncthreads();
  };
  auto add_mass = [&](int bin, unsigned long long w) {
    if (!w) return;
    const unsigned wl = (unsigned)w, old = atomicAdd(&s.lo[bin], wl);
    const unsigned wh = (unsigned)(w >> 32) + (old + wl < old ? 1u : 0u);
    if (wh) atomicAdd(&s.hi[bin], wh);
  };
  // s.sum: the bins' masses (what = 1), counts (0), or counts above the 32 bits of `lo`
  // (2), over the cluster: each CTA adds up some bins and tells all.
  auto combine = [&](int what) {
    if (ctas == 1) {
      __syncthreads();
      for (int i = tid; i < kSpBins; i += kSpThreads)
        s.sum[i] = what == 0 ? s.count[i] : s.lo[i] + ((unsigned long long)(what == 1 ? s.hi[i] : s.count[i]) << 32);
      __syncthreads();
      return;
    }
    cluster_sync();
    // the CTA's kSpBins / ctas bins, `team` neighbouring threads to each
    const int per = kSpBins / (int)ctas, b0 = (int)rank * per, team = max(1, kSpThreads / per), mate = tid % team;
    for (int i = b0 + tid / team; i < b0 + per; i += kSpThreads / team) {
      unsigned long long t = 0;
#pragma unroll 4
      for (uint32_t c = mate; c < ctas; c += team) {
        unsigned long long x;
        if (what == 0) {
          x = ld_cluster_u32(cluster_addr(&s.count[i], c));
        } else {
          x = ld_cluster_u32(cluster_addr(&s.lo[i], c));
          x += (unsigned long long)ld_cluster_u32(cluster_addr(what == 1 ? &s.hi[i] : &s.count[i], c)) << 32;
        }
        t += x;
      }
      for (int o = 1; o < team; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      for (uint32_t c = mate; c < ctas; c += team) st_cluster_u64(cluster_addr(&s.sum[i], c), t);
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
  // The first bin at which above + the running sum of `of` reaches the target:
  // s.found_bin, what lies above it: s.found_above, and all: s.found_total.
  auto find_bin = [&](unsigned long long above, unsigned long long target, auto&& of) {
    unsigned long long run[4];
    scan_bins(run, of);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned long long v = of(4 * tid + e);
      if (above + run[e] >= target && above + run[e] - v < target) {
        s.found_bin = 4 * tid + e;
        s.found_above = above + run[e] - v;
      }
    }
    if (tid == kSpThreads - 1) s.found_total = above + run[3];
    __syncthreads();
  };
  // bins of the first histogram: linear from the maximum down to the lowest value, or
  // to where nothing weighs
  const float bottom = fmaxf(key_float(lowest), m - kSpFar / sc.c);
  const float unit = (m - bottom) / (float)kSpBins, per_unit = fminf((float)kSpBins / (m - bottom), FLT_MAX);
  auto bin1 = [&](float v) { return (int)fminf((m - v) * per_unit, (float)(kSpBins - 1)); };
  // the bounds of two keys over the CTA's threads, in s.key_lo and s.key_hi
  auto bounds = [&](unsigned lo, unsigned hi) {
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicMin(&s.key_lo, lo);
      atomicMax(&s.key_hi, hi);
    }
    __syncthreads();
  };

  // One cut over all values, where the short ways failed: the smallest leading run of the
  // values above key `in` whose count or mass reaches `target` (it does).
  auto find_slowly = [&](bool mass, unsigned long long target, unsigned in) {
    unsigned khi = mkey, klo = 0;
    int shift = -1, want = -1;         // first level: linear in the value
    unsigned long long above = 0;      // what lies above the bin under search
    SpCut out{0u, ~0ull};
    for (int level = 0; level < 6; ++level) {
      clear(mass);
      for (int i = first + 4 * lane; i < last; i += 128) {
        const float4 v4 = load4(i, last);
        const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll 1
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
      find_bin(above, target, [&](int i) { return s.sum[i]; });
      const int bin = s.found_bin;
      above = s.found_above;
      if (bin < 0) return out;
      if (level > 0 && shift == 0) {
        // a single value: as many of its equals as the target takes
        const unsigned long long w = mass ? weight(key_float(khi - (unsigned)bin)) : 1ull;
        out.key = khi - (unsigned)bin;
        out.ties = w ? (target - above + w - 1) / w : 1;
        return out;
      }
      if (level == 0) {
        want = bin;
        unsigned lo_key = 0xffffffffu, hi_key = 0u;  // the bounds of the bin's keys
        for (int i = first + 4 * lane; i < last; i += 128) {
          const float4 v4 = load4(i, last);
          const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            const unsigned k = key_of(vs[e]);
            if (!(vs[e] >= -FLT_MAX) || k <= in || bin1(vs[e]) != want) continue;
            lo_key = min(lo_key, k);
            hi_key = max(hi_key, k);
          }
        }
        bounds(lo_key, hi_key);
        klo = s.key_lo;
        khi = s.key_hi;
        if (ctas > 1) {
          exchange(s, 1, klo, khi, rank, ctas);
          for (uint32_t c = 0; c < ctas; ++c) {
            klo = min(klo, (unsigned)s.board[1].a[c]);
            khi = max(khi, (unsigned)s.board[1].b[c]);
          }
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

  // ------------------------------------------------------ what is kept, run by run
  // The mass and the number of this run's values above the cut (with `from`: from it on),
  // and the number of those equal to it.
  auto sum_run = [&](unsigned least, bool from, int i0, int i1, unsigned long long& w, unsigned& c, unsigned& eq) {
    const float least_v = key_float(max(least, 0x00800000u));  // no finite value is below
    w = 0;
    c = eq = 0;
    each4(Ahead2{}, i0, i1, [&](const float4& v4, int, int) {
      if (!__any_sync(0xffffffffu, fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w)) >= least_v)) return;
      const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned k = vs[e] >= -FLT_MAX ? key_of(vs[e]) : 0u;
        const bool in = k > least || (from && k == least);
        SpWeight x = weight_parts(vs[e], sc, s.pow2);
        if (greedy) x = SpWeight{1u, 1u};
        if (in) {
          x.add_to(w);
          ++c;
        }
        eq += k == least;
      }
    });
    w = warp_sum(w);
    c = __reduce_add_sync(0xffffffffu, c);
    eq = __reduce_add_sync(0xffffffffu, eq);
  };
  // .. told to the leader
  auto tell_run = [&](unsigned long long w, unsigned c, unsigned eq, unsigned listed) {
    if (lane == 0) {
      st_cluster_u64(cluster_addr(&s.run_mass[mine], 0), w);
      st_cluster_u32(cluster_addr(&s.run_count[mine], 0), c);
      st_cluster_u32(cluster_addr(&s.run_equal[mine], 0), eq);
      st_cluster_u32(cluster_addr(&s.run_listed[mine], 0), listed);
    }
  };

  SpCut cut{0u, ~0ull};  // all
  bool listed = false;   // whether the border's neighbourhood is in lists
  unsigned long long above = 0, all = 0, target = 0;
  float lo = 0.f, hi = m;
  const bool by_k = top_k > 0 && (unsigned long long)top_k < finite, by_p = top_p < 1.f, floored = floor_key > 1u;
  const unsigned long long p = by_p ? fraction(top_p) : 0ull;
  auto share = [&](unsigned long long x) { return max(1ull, __umul64hi(x, p) + (x * p != 0 ? 1 : 0)); };  // ceil(p x)
  if (greedy) {
    cut.key = mkey;
    cut.ties = 1;
  } else if (by_k || by_p) {
    // ---- a bracket: without a sample, all values
    lo = bottom;
    // of the sample: the running sum (low word) and count (high word) at a thread's bins
    unsigned long long run[4];
    const int bits = 28 - (32 - __clz(a.slice / a.step));  // a weight's, so that the whole sample's sum fits 32
    const float floor_v = key_float(max(floor_key, 0x00800000u));
    // What min_p leaves out needs no list: a bracket that ends below its floor begins
    // there, and one that lies below it is empty, with all from the floor on above it.
    // Nothing that may be kept lies below it then.
    bool to_floor = false;
    auto at_floor = [&]() {
      to_floor = !by_k && floored && lo <= floor_v;
      if (!to_floor) return;
      lo = floor_v;
      if (hi < floor_v) {
        hi = key_float(floor_key - (floor_v == 0.f ? 2u : 1u));  // the first value below (0 is not above -0)
        lo = INFINITY;
      }
    };
    // The bracket about the bin at which the sample's mass (or count) reaches `goal`: the
    // values that lie kSpSide sampled ones before and behind.
    auto bracket = [&](float goal) {
      if (tid == 0) {
        s.bracket_hi = m;
        s.bracket_lo = kNone;
        s.found_above = ~0ull;  // its place in the sample
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned long long x = s.sum[4 * tid + e];
        const float now = by_k ? (float)(run[e] >> 32) : (float)(unsigned)run[e];
        const float was = by_k ? (float)((run[e] - x) >> 32) : (float)(unsigned)(run[e] - x);
        if (was < goal && now >= goal) s.found_above = run[e] >> 32;
      }
      __syncthreads();
      const unsigned long long at = s.found_above;
      if (at != ~0ull) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int b = 4 * tid + e;
          const unsigned long long here = run[e] >> 32, prev = (run[e] - s.sum[b]) >> 32;
          // the last bin that ends kSpSide before, the first that ends kSpSide behind
          if (b + 1 < kSpBins && here + kSpSide <= at && here + kSpSide + (s.sum[b + 1] >> 32) > at)
            s.bracket_hi = m - (float)(b + 1) * unit;
          if (b + 1 < kSpBins && here >= at + kSpSide && prev < at + kSpSide) s.bracket_lo = m - (float)(b + 1) * unit;
        }
      }
      __syncthreads();
      hi = by_k ? m : s.bracket_hi;  // (the first k are all listed)
      lo = fmaxf(bottom, s.bracket_lo);
    };
    if (sampled) {
      clear(true);
      for (int i = first + 4 * lane, b = 0; i < last; i += 128 * a.step, ++b) {
        const float4 v4 = sample[b * 32];
        const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!(vs[e] >= -FLT_MAX)) continue;
          const int b = bin1(vs[e]);
          atomicAdd(&s.count[b], 1u);
          if (!by_k) {
            // rounded up or down by the value's place, so that many small weights lose nothing on the whole
            const unsigned long long dither = (unsigned)(i + e) * 0x9e3779b1u & ((1u << (kSpTop - bits)) - 1u);
            const unsigned w = (unsigned)((weight(vs[e]) + dither) >> (kSpTop - bits));
            if (w) atomicAdd(&s.lo[b], w);
          }
        }
      }
      combine(2);
      scan_bins(run, [&](int i) { return s.sum[i]; });
      if (tid == kSpThreads - 1) s.warp_b[0] = (unsigned)run[3];
      __syncthreads();
      bracket(fmaxf(by_k ? (float)top_k / (float)a.step : top_p * (float)s.warp_b[0], 1e-30f));
    }
    const float sample_sum = sampled ? (float)s.warp_b[0] : 0.f;
    __syncthreads();

    // ---- all values: their sum, what lies above the bracket, and the lists
    for (int round = 0; round < kSpTries; ++round) {
      at_floor();
      unsigned long long w_below = 0, w_above = 0, w_list = 0;
      unsigned c_above = 0, n_list = 0;
      float* my_v = list_v + warp * cap;
      auto list = [&](float v) {  // if it lies in the bracket
        const bool in = v >= lo && v <= hi;
        const unsigned b = __ballot_sync(0xffffffffu, in), at = n_list + __popc(b & ((1u << lane) - 1));
        if (in && at < (unsigned)cap) my_v[at] = v;
        n_list += __popc(b);
      };
      if (by_k) {
        each4(Ahead4{}, first, last, [&](const float4& v4, int, int) {
          if (!__any_sync(0xffffffffu, fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w)) >= lo)) return;
          list(v4.x);
          list(v4.y);
          list(v4.z);
          list(v4.w);
        });
      } else {
        each4(Ahead2{}, first, last, [&](const float4& v4, int, int) {
          const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const SpWeight x = weight_parts(vs[e], sc, s.pow2);
            if (vs[e] > hi) {
              x.add_to(w_above);
              ++c_above;
            } else {
              x.add_to(w_below);
            }
            list(vs[e]);
          }
        });
        __syncwarp();
        for (unsigned i = lane; i < min(n_list, (unsigned)cap); i += 32) w_list += weight(my_v[i]);
      }
      unsigned long long w_all = warp_sum(w_below + w_above);
      w_above = warp_sum(w_above);
      w_list = warp_sum(w_list);
      c_above = __reduce_add_sync(0xffffffffu, c_above);
      // the row's sums (a list that ran over is told by a count beyond any)
      const unsigned long long n_told = n_list > (unsigned)cap ? 1ull << 40 : n_list;
      if (lane == 0) {
        s.part[0][warp] = w_all;
        s.part[1][warp] = w_above;
        s.part[2][warp] = w_list;
        s.part[3][warp] = n_told;
      }
      __syncthreads();
      unsigned long long t[4];
      const int x = round % 2 ? 0 : 2;  // boards in turns: the others may still read the last ones
      if (warp == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          t[q] = warp_sum(lane < kSpWarps ? s.part[q][lane] : 0ull);
          if (lane < (int)ctas) st_cluster_u64(cluster_addr(q % 2 ? &s.board[x + q / 2].b[rank] : &s.board[x + q / 2].a[rank], lane), t[q]);
        }
      }
      if (ctas > 1) cluster_sync();
      else __syncthreads();
#pragma unroll
      for (int q = 0; q < 4; ++q) t[q] = 0;
      for (uint32_t c = 0; c < ctas; ++c) {
        t[0] += s.board[x].a[c];
        t[1] += s.board[x].b[c];
        t[2] += s.board[x + 1].a[c];
        t[3] += s.board[x + 1].b[c];
      }
      const unsigned long long t_all = t[0], t_above = t[1], t_list = t[2], t_n = t[3];
      above = t_above;
      all = t_all;
      if (by_k) {
        listed = t_n < (1ull << 40) && t_n >= (unsigned long long)top_k;
      } else {
        target = share(all);
        // (the border lies in the bracket, or below the floor, where it is of no matter; a
        // list that ran over is not added up)
        const bool border = above < target && (above + t_list >= target || to_floor);
        listed = border && t_n < (1ull << 40);
        if (!border && sampled && round + 1 < kSpTries) {
          // the sample's own sums from the nearer end of the bracket on
          const bool before = above >= target;
          const float edge = before ? hi : fminf(lo, hi);
          const int b = min(kSpBins - 1, max(0, (int)rintf((m - edge) / unit)));  // the first bin behind the edge
          if (b / 4 == tid) s.found_total = (unsigned)(run[b % 4] - s.sum[b]);
          __syncthreads();
          const float at_edge = (float)s.found_total;
          const float off = before ? -(float)(above - target) : (float)(target - above - t_list);
          __syncthreads();
          bracket(fminf(fmaxf(at_edge + off * exp2f((float)(bits - kSpTop)) / (float)a.step, 1e-30f), sample_sum));
          continue;
        }
      }
      if (listed) {
        tell_run(w_above, c_above, 0u, n_list);
        if (rank > 0) {
          const uint32_t to = cluster_addr(list_v + mine * cap, 0);
          for (unsigned i = lane; i < n_list; i += 32) st_cluster_u32(to + 4 * i, __float_as_uint(my_v[i]));
        }
      }
      break;
    }
    if (!listed) {
      // ---- the long way
      if (by_k) cut = find_slowly(false, (unsigned long long)top_k, 0u);
      if (by_p) {
        SpCut c{0u, ~0ull};
        unsigned long long sum = all, eq_w = 0;
        if (by_k) {
          unsigned long long w;
          unsigned n, eq;
          sum_run(cut.key, false, first, last, w, n, eq);
          unsigned long long t = lane == 0 ? w : 0, none = 0;
          cta_sum(s, t, none);
          if (ctas > 1) {
            cluster_sync();
            exchange(s, 3, t, 0, rank, ctas);
            t = 0;
            for (uint32_t x = 0; x < ctas; ++x) t += s.board[3].a[x];
          }
          eq_w = weight(key_float(cut.key));
          sum = t + cut.ties * eq_w;
          target = share(sum);
          if (t < target) {
            c.key = cut.key;
            c.ties = eq_w ? (target - t + eq_w - 1) / eq_w : 1;
          }
        }
        if (!c.key) c = find_slowly(true, target, cut.key);
        if (c.key) cut = c;
      }
    }
  }

  if (!listed) {
    const bool tied = cut.key && cut.ties != ~0ull && cut.key >= floor_key;
    unsigned long long w;
    unsigned c, eq;
    sum_run(tied ? cut.key : max(cut.key, floor_key), !tied, first, last, w, c, eq);
    tell_run(w, c, tied ? eq : 0u, 0u);
  }
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  if (rank > 0) return;

  // ================================================================= the leader
  // a team of threads for every run's list (a warp at most: there are 16 runs at least)
  const int team = kSpThreads / runs, my_run = tid / team, mate = tid % team;
  // two values at a time, the second with key 0 where there is none
  auto each_listed = [&](auto&& f) {
    const int n = (int)s.run_listed[my_run];
    for (int i = mate; i < n; i += 2 * team) {
      const float* at = list_v + my_run * cap + i;
      const float v0 = at[0], v1 = i + team < n ? at[team] : kNone;
      f(v0, v1, key_of(v0), v1 >= -FLT_MAX ? key_of(v1) : 0u);
    }
  };
  // The inclusive running sum over the CTA's threads
  auto scan = [&](unsigned long long x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s.warp_a[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += s.warp_a[w];
    return x;
  };
  if (listed) {
    // One cut among the listed values above key `in`: bins linear in the value, and where
    // a bin holds too many different ones, over the bits of their keys.
    auto find_listed = [&](bool mass, unsigned long long goal, unsigned long long over, unsigned in, SpCut& out) {
      constexpr int kBins = kSpThreads;  // a thread's each
      const float scale = fminf((float)kBins / (hi - lo), FLT_MAX);
      unsigned khi = 0, klo = 0;
      int shift = -1;
      auto bin_of = [&](float v, unsigned k) {
        if (shift < 0) return (int)fminf((hi - v) * scale, (float)(kBins - 1));
        return k > khi || k < klo ? -1 : (int)((khi - k) >> shift);
      };
      for (int level = 0; level < 6; ++level) {
        __syncthreads();
        s.count[tid] = s.lo[tid] = s.hi[tid] = 0u;
        if (tid == 0) {
          s.found_bin = -1;
          s.nkeys = 0;
          s.key_lo = 0xffffffffu;
          s.key_hi = 0;
        }
        __syncthreads();
        each_listed([&](float v0, float v1, unsigned k0, unsigned k1) {
          const int b0 = k0 > in ? bin_of(v0, k0) : -1, b1 = k1 > in ? bin_of(v1, k1) : -1;
          const unsigned long long w0 = mass ? weight(v0) : 0ull, w1 = mass ? weight(v1) : 0ull;
          if (b0 >= 0) {
            if (mass) add_mass(b0, w0);
            else atomicAdd(&s.count[b0], 1u);
          }
          if (b1 >= 0) {
            if (mass) add_mass(b1, w1);
            else atomicAdd(&s.count[b1], 1u);
          }
        });
        __syncthreads();
        const unsigned long long mine_w = mass ? s.lo[tid] + ((unsigned long long)s.hi[tid] << 32) : (unsigned long long)s.count[tid];
        const unsigned long long upto = over + scan(mine_w);
        if (upto >= goal && upto - mine_w < goal) {
          s.found_bin = tid;
          s.found_above = upto - mine_w;
        }
        __syncthreads();
        const int bin = s.found_bin;
        if (bin < 0) return;
        over = s.found_above;
        auto take = [&](float v, unsigned k) {
          if (k <= in || bin_of(v, k) != bin) return;
          const unsigned at = atomicAdd(&s.nkeys, 1u);
          atomicMin(&s.key_lo, k);
          atomicMax(&s.key_hi, k);
          if (at < kSpKeys) s.keys[at] = k;
        };
        each_listed([&](float v0, float v1, unsigned k0, unsigned k1) {
          take(v0, k0);
          take(v1, k1);
        });
        __syncthreads();
        klo = s.key_lo;
        khi = s.key_hi;
        const unsigned n = s.nkeys;
        if (klo == khi) {
          const unsigned long long w = mass ? weight(key_float(klo)) : 1ull;
          out.key = klo;
          out.ties = (goal - over + w - 1) / w;
          return;
        }
        if (n <= kSpKeys) {
          // compared with one another; the weights lie where the cluster's sums were
          if (tid < (int)n) s.sum[tid] = mass ? weight(key_float(s.keys[tid])) : 1ull;
          __syncthreads();
          if (tid < (int)n) {
            const unsigned k = s.keys[tid];
            unsigned long long before = over, same = 0;
#pragma unroll 4
            for (unsigned i = 0; i < n; ++i) {
              const unsigned o = s.keys[i];
              if (o > k) before += s.sum[i];
              same += o == k;
            }
            const unsigned long long w = s.sum[tid];
            if (before < goal && before + same * w >= goal) s.cut = SpCut{k, (goal - before + w - 1) / w};  // (equal ones agree)
          }
          __syncthreads();
          out = s.cut;
          return;
        }
        shift = 0;
        while (((khi - klo) >> shift) >= kBins) ++shift;
      }
    };
    if (by_k) {
      find_listed(false, (unsigned long long)top_k, 0, 0u, cut);
      if (by_p) {
        unsigned long long w = 0, none = 0;
        each_listed([&](float v0, float v1, unsigned k0, unsigned k1) {
          const unsigned long long w0 = weight(v0), w1 = weight(v1);
          w += (k0 > cut.key ? w0 : 0ull) + (k1 > cut.key ? w1 : 0ull);
        });
        cta_sum(s, w, none);
        const unsigned long long w_tie = weight(key_float(cut.key)), goal = share(w + cut.ties * w_tie);
        if (w >= goal) find_listed(true, goal, 0, cut.key, cut);
        else cut.ties = w_tie ? (goal - w + w_tie - 1) / w_tie : 1;
      }
    } else {
      find_listed(true, target, above, 0u, cut);
    }
  }
  const bool tied = cut.key && cut.ties != ~0ull && cut.key >= floor_key;
  const unsigned least = tied ? cut.key : max(cut.key, floor_key);
  // ---- what is kept of each run (in its team's first thread), and the run that holds
  // the border; equal values are taken in the order of the runs
  const unsigned long long w_tie = tied ? weight(key_float(cut.key)) : 0ull;
  unsigned long long run_w = 0, run_c = 0, run_eq = 0;
  if (listed) {
    const unsigned above_it = tied ? least : least - 1u;
    each_listed([&](float v0, float v1, unsigned k0, unsigned k1) {
      const unsigned long long w0 = weight(v0), w1 = weight(v1);
      run_w += (k0 > above_it ? w0 : 0ull) + (k1 > above_it ? w1 : 0ull);
      run_c += (k0 > above_it) + (k1 > above_it);
      run_eq += (tied && k0 == least) + (tied && k1 == least);
    });
    for (int o = 1; o < team; o <<= 1) {
      run_w += __shfl_xor_sync(0xffffffffu, run_w, o);
      run_c += __shfl_xor_sync(0xffffffffu, run_c, o);
      run_eq += __shfl_xor_sync(0xffffffffu, run_eq, o);
    }
  } else {
    run_eq = s.run_equal[my_run];
  }
  run_w = mate == 0 ? run_w + s.run_mass[my_run] : 0;
  run_c = mate == 0 ? run_c + s.run_count[my_run] : 0;
  run_eq = mate == 0 ? run_eq : 0;
  {
    const unsigned long long ties = tied ? cut.ties : 0, upto = scan(run_eq), had = min(ties, upto - run_eq);
    run_eq = min(ties, upto) - had;  // from here on: how many of them are kept
    run_w += run_eq * w_tie;
    if (tid == 0) s.found_bin = -1;
    const unsigned long long w_upto = scan(run_w);
    const unsigned c = __reduce_add_sync(0xffffffffu, (unsigned)(run_c + run_eq));
    if (lane == 0) s.part[0][warp] = c;
    if (tid == kSpThreads - 1) s.found_total = w_upto;
    __syncthreads();
    if (warp == 0 && a.kept) {
      const unsigned all_c = __reduce_add_sync(0xffffffffu, lane < kSpWarps ? (unsigned)s.part[0][lane] : 0u);
      if (lane == 0) a.kept[row] = (int)all_c;
    }
    const unsigned long long goal = __umul64hi(s.found_total, fraction(u));  // the first running sum above it
    if (goal >= w_upto - run_w && goal < w_upto) {
      s.found_bin = my_run;
      s.found_above = w_upto - run_w;
      s.run_equal[my_run] = (unsigned)run_eq;
    }
  }
  __syncthreads();
  const int r = s.found_bin;
  if (r < 0) {  // no run is indexed that the sums do not name: the row is told as one that cannot be drawn from
    if (tid == 0) {
      a.token[row] = -1;
      if (a.logprob) a.logprob[row] = __uint_as_float(0x7fc00000u);
      if (a.kept) a.kept[row] = 0;
    }
    return;
  }
  const int f = run_first(r), l = run_last(r);
  const unsigned long long total = s.found_total, goal = __umul64hi(total, fraction(u));
  unsigned long long now = s.found_above, left = s.run_equal[r];
  // ---- a piece of it for each warp, and the piece that holds the border by its warp
  const int piece = ((l - f + kSpWarps - 1) / kSpWarps + 127) / 128 * 128, i0 = min(l, f + warp * piece), i1 = min(l, i0 + piece);
  unsigned long long w;
  unsigned c, eq;
  sum_run(least, !tied, i0, i1, w, c, eq);
  if (lane == 0) {
    s.warp_a[warp] = w;
    s.warp_b[warp] = tied ? eq : 0u;
  }
  __syncthreads();
  for (int x = 0; x < warp; ++x) {
    const unsigned long long take = min(left, s.warp_b[x]);
    now += s.warp_a[x] + take * w_tie;
    left -= take;
  }
  if (goal < now || goal >= now + w + min(left, s.warp_b[warp]) * w_tie) return;
  for (int i = i0 + 4 * lane; i - 4 * lane < i1; i += 128) {
    const float4 v4 = i < i1 ? load4(i, i1) : make_float4(kNone, kNone, kNone, kNone);
    const float vs[4] = {v4.x, v4.y, v4.z, v4.w};
    unsigned long long ws[4], sum = 0;
    unsigned equal = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned k = vs[e] >= -FLT_MAX ? key_of(vs[e]) : 0u;
      ws[e] = k > least || (!tied && k == least) ? weight(vs[e]) : 0ull;
      equal |= (tied && k == least ? 1u : 0u) << e;
    }
    // the equal ones' places
    unsigned upto = __popc(equal);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    unsigned long long place = upto - __popc(equal);
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
    unsigned long long at = now + inc - sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (ws[e] && goal >= at && goal < at + ws[e]) {
        a.token[row] = i + e;
        if (a.logprob) {
          // a likely token's is taken from what the others weigh, so that it is exact near 0 too
          const unsigned long long rest = total - ws[e];
          a.logprob[row] = rest < ws[e] ? ln_share(rest, ws[e])
                                        : (float)((((double)vs[e] - (double)sc.base) * ((double)sc.c + (double)sc.clo) -
                                                   log2_of(total, s.pow2) + (kSpTop - sc.nref)) * 0.69314718055994530942);
        }
      }
      at += ws[e];
    }
    left -= min(left, (unsigned long long)__shfl_sync(0xffffffffu, upto, 31));
    now += __shfl_sync(0xffffffffu, inc, 31);
    if (now > goal) return;
  }
}

// CTAs of a row's cluster: slices of 65536 values at most, of which a run's sample fits its
// place (256 rows of 262144: 4 CTAs 305 us, 8 347, 16 502), shorter ones of 2048 values at
// least while that gives every SM no more than one CTA (8 rows of 262144: 16 CTAs 36 us, 8
// 40, 4 53), and of 16384 up to two (64 rows of 151936: 4 CTAs 60 us, 8 78; 32 of 50257:
// 4 CTAs 34, 2 44, 8 37; 160 of 50257: 1 CTA 72, 2 81).
int sample_ctas(int R, int V) {
  int c = 1;
  while (c < kSpMaxCluster && (int64_t)c * 65536 < V) c *= 2;
  while (c < kSpMaxCluster) {
    const int64_t all = (int64_t)R * c * 2, least = all <= kTargetCtas ? 2048 : 16384;
    if (all > 2 * kTargetCtas || V < 2 * c * least) break;
    c *= 2;
  }
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
  const int ctas = sample_ctas(R, V);
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
  a.run4 = cdiv(cdiv(V, ctas * kSpWarps * 4), 32) * 32;
  a.slice = a.run4 * 4 * kSpWarps;
  a.step = a.slice >= 32768 ? 8 : a.slice >= 16384 ? 4 : a.slice >= 8192 ? 2 : 1;
  a.bf16 = bf16 != 0;
  a.temperature_all = how->temperature_all;
  a.top_p_all = how->top_p_all;
  a.min_p_all = how->min_p_all;
  a.top_k_all = how->top_k_all;
  cudaError_t e = set_smem_once<sample_kernel>(kSpSmem);
  if (e == cudaSuccess) e = allow_large_clusters();
  if (e != cudaSuccess) return DG_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(R, ctas);
  cfg.blockDim = dim3(kSpThreads);
  cfg.dynamicSmemBytes = kSpSmem;
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

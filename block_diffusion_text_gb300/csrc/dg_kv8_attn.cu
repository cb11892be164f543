// Attention over the 8-bit prefix cache for few query rows per kv head (single
// tokens, calls of few tiles, head dim 32), and the merge of the parts.
//
// A warp is a worker: it streams its share of key tiles through a ring of its
// own in shared memory (TMA, no barrier shared with other warps) and keeps
// queries, running maximum and sum, and the output of 8 NT rows in registers.
// Work for single tokens is bound by the bytes of the cache, so what counts is
// loads in flight, warps to cover each other's latencies, and few instructions
// per code:
//  - Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that
//    keys and output columns fill the 16 rows of mma.sync m16n8k16 and the
//    query rows its 8 columns: one token's group of up to 8 heads costs half
//    the MMAs, registers and exponentials of the untransposed form.
//  - The codes go from shared memory into the MMA fragments in one conversion
//    (two E4M3 to two f16, exact).  The fragments' index maps make that
//    possible: the sum over the head dim may run in any order, so lane t of a
//    quad owns the contiguous quarter t of a key row; the output columns may
//    be dealt in any order, so lane group g owns the contiguous eighth g of a
//    value row.  (E4M3 MMAs of this shape would spare the conversion of the
//    keys; with operands that change they took longer, 36 against 14 cycles
//    each in this loop, measured.)
//  - Block scales never touch the codes.  The key scale joins the softmax
//    factor; the value scale 2^e joins the exponent of the probability,
//    p' = 2^(s + e - m), so that P' V sums codes, with m the running maximum of
//    s + e; the row sum takes p' 2^-e back.
//  - Queries enter as f16 scaled by a power of two per row (exact for elements
//    down to 2^-27 of the row's largest).  p' is rounded to f16 (2^-11 of its
//    value; 2^-33 of the largest at least, with the headroom of 2^8 below):
//    an eighth of the rounding of the bf16 output.
// New tokens' bf16 keys and values keep their exponent range: bf16 MMAs, P
// split into two bf16 parts (2^-17).
// Measured: one token of 4 sequences over 131072 rows of 8 heads 166 to 169 us (6.4
// TB/s, 94 % of the measured copy rate), of 32 sequences of 0 to 8192 rows 48 us (5.2
// TB/s; the start and the merge take some 8 us), of one over 2048 rows 7.4 us (11
// with one CTA to a kv head; a launch takes 2).
#include <cfloat>

#include "dg_kv8.cuh"

namespace dg {
namespace {

constexpr float kHeadroom = 8.0f;  // p' of a row's maximum is 2^8 ..
constexpr float kLazy = 4.0f;      // .. to 2^12: the maximum is followed when it grows by more than 2^4
constexpr int kStep = 32;          // keys per step
constexpr int kMT = kStep / 16;    // their m-tiles

// W warps with a ring of kStages steps each.
template <int HD, int W>
struct Ring {
  static constexpr int kHalf = kStep * HD;     // codes of K (or V) of one step
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = (W == 8 ? 24576 : 16384) / kStage;
  static constexpr int kWarp = kStages * kStage;
  static constexpr int oMl = W * kWarp;           // float2 [warps][32 rows]
  static constexpr int oBar = oMl + W * 32 * 8;   // mbarriers [warps][stages]
  static constexpr int oJoin = oBar + W * kStages * 8 + 16;  // the CTA's merged parts: float [rows][HD],
  static constexpr int kJoin = (W == 8 ? 2048 : 1024) * 4;   // as many as kv8_mma_warps allows rows,
  static constexpr int kSmem = oJoin + kJoin + 32 * 8;       // and float2 [32 rows]
  static_assert(oJoin % 16 == 0 && kSmem <= 232448, "shared memory of one CTA");
};

// The MMAs without the order that volatile asm keeps: the scheduler may move
// conversions and independent products between dependent ones.
DG_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
DG_DEV void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8x8 matrix of 16-bit elements transposed across the warp: an accumulator
// fragment's rows become the columns of a B fragment.
DG_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// Bounded wait of a whole warp, one try first and the loops out of line.
__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  return mbar_wait_warp(bar, parity, status, abort);
}
DG_DEV bool wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_more(bar, parity, status, abort);
}

// Rows 2t and 2t + 1 of each n-tile; o: columns g HD / 8 + 2 i (elements 0, 1)
// and + 2 i + 1 (elements 2, 3).
template <int HD, int NT>
struct Acc {
  float o[NT][HD / 16][4];
  float m[NT][2], l[NT][2];
};

// One step's scores to probabilities: s (raw products; keys 16 mt + g and + 8,
// rows 2t and 2t + 1 of each n-tile) become p' = 2^(s c + ev - m + headroom).
template <int HD, int NT>
DG_DEV void softmax_step(float (&s)[kMT][NT][4], const float (&c)[NT][2], float ev, float inv_ev, Acc<HD, NT>& acc) {
  float mx[NT][2];
  bool need = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
      for (int mt = 1; mt < kMT; ++mt) v = fmax3(v, s[mt][nt][e], s[mt][nt][2 + e]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
      mx[nt][e] = fmaf(v, c[nt][e], ev);
      need |= mx[nt][e] > acc.m[nt][e] + kLazy;
    }
  }
  if (__any_sync(0xffffffffu, need)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float corr[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(mx[nt][e], acc.m[nt][e]);
        corr[e] = mn > acc.m[nt][e] ? ex2_approx(acc.m[nt][e] - mn) : 1.0f;
        acc.m[nt][e] = mn;
        acc.l[nt][e] *= corr[e];
      }
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc.o[nt][i][k] *= corr[k & 1];
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float m = acc.m[nt][e];
      const float off = ev - (m == -INFINITY ? 0.0f : m - kHeadroom);
      float sum = 0.f;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p = ex2_approx(fmaf(s[mt][nt][2 * h + e], c[nt][e], off));
          s[mt][nt][2 * h + e] = p;
          sum += p;
        }
      }
      acc.l[nt][e] = fmaf(sum, inv_ev, acc.l[nt][e]);
    }
  }
}

// Parts of 4 N output columns and the row sum, on the maximum M of all parts.
template <int N>
struct Kv8Sum {
  float l = 0.f;
  float4 v[N] = {};
  // x: the part's columns, the next four `step` further
  DG_DEV void add(const float2& ml, float M, const float4* x, size_t step) {
    float4 p[N];
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = x[i * step];
    const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
    l = fmaf(w, ml.y, l);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i].x = fmaf(w, p[i].x, v[i].x);
      v[i].y = fmaf(w, p[i].y, v[i].y);
      v[i].z = fmaf(w, p[i].z, v[i].z);
      v[i].w = fmaf(w, p[i].w, v[i].w);
    }
  }
  DG_DEV void add(const Kv8Sum& s) {
    l += s.l;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i].x += s.v[i].x;
      v[i].y += s.v[i].y;
      v[i].z += s.v[i].z;
      v[i].w += s.v[i].w;
    }
  }
  DG_DEV void store(__nv_bfloat16* dst) const {
    const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < N; ++i)
      *reinterpret_cast<uint2*>(dst + 4 * i) =
          make_uint2(pack_bf16(v[i].x * inv, v[i].y * inv), pack_bf16(v[i].z * inv, v[i].w * inv));
  }
};

// Loads from the shared memory of a CTA of the cluster.
DG_DEV float2 ld_cluster_v2(uint32_t caddr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(caddr) : "memory");
  return v;
}
DG_DEV float4 ld_cluster_v4(uint32_t caddr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(caddr)
               : "memory");
  return v;
}

// NB bytes of a fragment slice from shared memory.
template <int NB>
DG_DEV void lds(uint32_t* w, const uint8_t* p) {
  if constexpr (NB == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (NB == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

template <int HD, int NT, int W>
__global__ void __launch_bounds__(32 * W, 1)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, Kv8AttnArgs a,
                    float scale_log2) {
  using R = Ring<HD, W>;
  constexpr int SL = HD / 4;   // elements of a key row per quad lane
  constexpr int KS = HD / 16;  // k16 steps of K Q^T, m-tiles of V^T P^T
  constexpr int NV = HD / 8;   // columns of a value row per lane group
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {  // uniform over the CTA
    if (threadIdx.x == 0) atomicExch(a.status, kStatusTimeout);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  uint8_t* ring = smem + warp * R::kWarp;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + R::oBar) + warp * R::kStages;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + R::oBar + W * R::kStages * 8);
  const int worker = warp * gridDim.x + blockIdx.x;  // consecutive shares on different SMs
  if (threadIdx.x == 0) {
    *abort = 0;
    tma_prefetch(&mK);
    tma_prefetch(&mV);
  }
  if (lane == 0) {
    for (int i = 0; i < R::kStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();  // the next kernel (the merge, or with clusters any) waits for this one's completion all the same

  if (worker == 0) {
    for (int b = lane; b < a.B; b += 32)
      if (a.len[b] < 0 || a.len[b] > a.cap) atomicExch(a.status, kStatusCapacity);
  }
  const int rank = a.cluster ? (int)blockIdx.x % a.cluster : 0;
  int lead = 0;  // first warp of the warp's group
  int w = a.cluster ? (int)blockIdx.x / a.cluster : 0;  // a cluster's unit, or a group's
  if (a.cluster && a.group < W) {
    lead = warp / a.group * a.group;
    w = w * (W / a.group) + lead / a.group;  // behind the last unit for groups without any
  }
  int w1 = w + 1;
  Kv8Plan plan{};
  int2 from = make_int2(0, 0);
  if (!a.cluster) {
    plan = kv8_plan(a);
    w1 = (int)min((long long)plan.total, (worker + 1ll) * plan.share);
    w = (int)min((long long)w1, (long long)worker * plan.share);
  }
  const int grp_rows = a.Hq / a.Hkv * a.C, row_tiles = a.units / a.Hkv;
  int slot = 0, par = 0;  // the ring's stage to read next, and its barrier's parity
  bool ok = true;

  while (w < w1 && ok) {
    Kv8Piece p;
    if (a.cluster) {
      p.b = w / a.units;
      p.len = p.b < a.B ? kv8_len(a, p.b) : 0;
      p.nt = p.b < a.B ? kv8_tiles(a, p.len) : 0;
      p.unit = w - p.b * a.units;
      const int n = a.group * a.cluster, chunk = (p.nt + n - 1) / n;
      p.t0 = min(((warp - lead) * a.cluster + rank) * chunk, p.nt);
      p.t1 = min(p.t0 + chunk, p.nt);
    } else {
      p = kv8_piece(a, plan, from, w, w1);
      w += p.cost;
      if (p.t1 <= p.t0) continue;
    }
    const int t0 = p.t0, t1 = p.t1;
    const int hk = p.unit / row_tiles, row0 = p.unit % row_tiles * (8 * NT);
    const int ntc = (p.len + kKv8Block - 1) / kKv8Block;
    const int tc1 = min(t1, ntc);  // cached tiles of the piece end here
    const size_t bh = (size_t)p.b * a.Hkv + hk;
    const uint8_t* Ke = a.Ke + bh * a.nblk;
    const uint8_t* Ve = a.Ve + bh * a.nblk;
    const int nsteps = max(tc1 - t0, 0) * (kKv8Block / kStep);

    // Step i of the piece into the ring, `ahead` stages past the one to read next.
    auto issue = [&](int i, int ahead) {
      if (i < nsteps && lane == 0) {
        int st = slot + ahead;
        if (st >= R::kStages) st -= R::kStages;
        uint8_t* dst = ring + st * R::kStage;
        const int row = (int)bh * a.cap + t0 * kKv8Block + i * kStep;
        mbar_arrive_expect_tx(&full[st], R::kStage);
        tma_load_2d(dst, &mK, &full[st], 0, row);
        tma_load_2d(dst + R::kHalf, &mV, &full[st], 0, row);
      }
    };
#pragma unroll
    for (int i = 0; i < R::kStages; ++i) issue(i, i);

    // Queries: row g of each n-tile, elements t SL + 4 j .. + 3 of step j, as f16
    // on the power-of-two scale of the row.
    uint32_t qf[NT][KS][2];
    int qx[NT][2];    // exponents of rows 2t and 2t + 1
    int qi[NT][2];    // their tokens' positions among the new ones
    const __nv_bfloat16* qrow[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      const bool there = r < grp_rows && p.b < a.B;
      qrow[nt] = there ? reinterpret_cast<const __nv_bfloat16*>(a.q) + (bh * grp_rows + r) * HD + t * SL : nullptr;
      uint2 raw[KS];
      unsigned top = 0;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        raw[j] = there ? *reinterpret_cast<const uint2*>(qrow[nt] + 4 * j) : make_uint2(0, 0);
        top = __vmaxu2(top, __vmaxu2(raw[j].x & 0x7fff7fffu, raw[j].y & 0x7fff7fffu));
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int x = top == 0 ? 0 : max((int)(top >> 7) - 127 - 13, -127);
      const float f = pow2i(-x);
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        qf[nt][j][0] = pack_f16(__uint_as_float(raw[j].x << 16) * f, __uint_as_float(raw[j].x & 0xffff0000u) * f);
        qf[nt][j][1] = pack_f16(__uint_as_float(raw[j].y << 16) * f, __uint_as_float(raw[j].y & 0xffff0000u) * f);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qx[nt][e] = __shfl_sync(0xffffffffu, x, (2 * t + e) * 4);
        qi[nt][e] = (row0 + nt * 8 + 2 * t + e) % a.C;
      }
    }
    Acc<HD, NT> acc;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        acc.m[nt][e] = -INFINITY;
        acc.l[nt][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc.o[nt][i][k] = 0.f;
    }

    int ke_next = 0, ve_next = 0, ke = 0, ve = 0, ve_top = kKv8Emin;
    if (nsteps > 0) {
      ke_next = Ke[t0];
      ve_next = Ve[t0];
    }
#pragma unroll 1
    for (int i = 0; i < nsteps; ++i) {
      if (i % (kKv8Block / kStep) == 0) {
        ke = ke_next - kKv8Bias;
        ve = ve_next - kKv8Bias;
        ve_top = max(ve_top, ve);
        const int nx = t0 + i / (kKv8Block / kStep) + 1;
        if (nx < tc1) {
          ke_next = Ke[nx];
          ve_next = Ve[nx];
        }
      }
      if (!(ok = wait(&full[slot], par, a.status, abort))) break;
      const int valid = p.len - (t0 * kKv8Block + i * kStep);
      if (valid > 0) {
        const uint8_t* sk = ring + slot * R::kStage;
        const uint8_t* sv = sk + R::kHalf;
        float s[kMT][NT][4];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[mt][nt][k] = 0.f;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          uint32_t kw[2][SL / 4];  // keys 16 mt + g and + 8
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = 16 * mt + 8 * h + g;
            if constexpr (HD == 128) {
              lds<16>(&kw[h][0], sk + r * HD + (((2 * t) ^ swz<HD>(r)) * 16));
              lds<16>(&kw[h][4], sk + r * HD + (((2 * t + 1) ^ swz<HD>(r)) * 16));
            } else if constexpr (HD == 64) {
              lds<16>(&kw[h][0], sk + r * HD + ((t ^ swz<HD>(r)) * 16));
            } else {
              lds<8>(&kw[h][0], sk + r * HD + (((t / 2) ^ swz<HD>(r)) * 16) + (t & 1) * 8);
            }
          }
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            uint32_t ka[4];
            e4m3x4_f16x4(kw[0][j], ka[0], ka[2]);
            e4m3x4_f16x4(kw[1][j], ka[1], ka[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(s[mt][nt], ka, qf[nt][j][0], qf[nt][j][1]);
          }
        }
        if (valid < kStep) {
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (16 * mt + g + 8 * (k >> 1) >= valid) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[mt][nt][k] = -INFINITY;
              }
        }
        float c[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) c[nt][e] = scale_log2 * pow2i(qx[nt][e] + ke);
        softmax_step<HD, NT>(s, c, (float)ve, pow2i(-ve), acc);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          uint32_t vw[4][NV / 4];  // keys 2t, 2t + 1, 2t + 8, 2t + 9; the lane group's columns
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 16 * mt + 2 * t + (q & 1) + 8 * (q >> 1);
            if constexpr (HD == 128)
              lds<16>(vw[q], sv + r * HD + ((g ^ swz<HD>(r)) * 16));
            else if constexpr (HD == 64)
              lds<8>(vw[q], sv + r * HD + (((g / 2) ^ swz<HD>(r)) * 16) + (g & 1) * 8);
            else
              lds<4>(vw[q], sv + r * HD + (((g / 4) ^ swz<HD>(r)) * 16) + (g & 3) * 4);
            if (valid < kStep && r >= valid) {  // what lies behind the sequence never enters an MMA
#pragma unroll
              for (int n = 0; n < NV / 4; ++n) vw[q][n] = 0;
            }
          }
          uint32_t pb[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            pb[nt][0] = transpose8x8(pack_f16(s[mt][nt][0], s[mt][nt][1]));
            pb[nt][1] = transpose8x8(pack_f16(s[mt][nt][2], s[mt][nt][3]));
          }
#pragma unroll
          for (int i = 0; i < KS; ++i) {  // two columns of four keys from two byte interleaves
            const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
            uint32_t va[4];
            e4m3x4_f16x4(__byte_perm(vw[0][i / 2], vw[1][i / 2], sel), va[0], va[1]);
            e4m3x4_f16x4(__byte_perm(vw[2][i / 2], vw[3][i / 2], sel), va[2], va[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(acc.o[nt][i], va, pb[nt][0], pb[nt][1]);
          }
        }
      }
      __syncwarp();  // the stage may be filled again
      issue(i + R::kStages, 0);
      if (++slot == R::kStages) {
        slot = 0;
        par ^= 1;
      }
    }

    // New tokens, in bf16, straight from global memory: a call has few of
    // them where this kernel is used.
    const __nv_bfloat16* kn = reinterpret_cast<const __nv_bfloat16*>(a.kn) + bh * a.C * HD;
    const __nv_bfloat16* vn = reinterpret_cast<const __nv_bfloat16*>(a.vn) + bh * a.C * HD;
    unsigned vn_top = 0;
#pragma unroll 1
    for (int key0 = (max(t0, ntc) - ntc) * kKv8Block, end = min((t1 - ntc) * kKv8Block, a.C); key0 < end;
         key0 += kStep) {
      float s[kMT][NT][4];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[mt][nt][k] = 0.f;
        const int kg = key0 + 16 * mt + g;
#pragma unroll
        for (int j = 0; j < KS; j += 2) {
          uint4 k0 = make_uint4(0, 0, 0, 0), k1 = k0;
          if (kg < a.C) k0 = *reinterpret_cast<const uint4*>(kn + (size_t)kg * HD + t * SL + 4 * j);
          if (kg + 8 < a.C) k1 = *reinterpret_cast<const uint4*>(kn + (size_t)(kg + 8) * HD + t * SL + 4 * j);
          const uint32_t a0[4] = {k0.x, k1.x, k0.y, k1.y}, a1[4] = {k0.z, k1.z, k0.w, k1.w};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 qv = qrow[nt] ? *reinterpret_cast<const uint4*>(qrow[nt] + 4 * j) : make_uint4(0, 0, 0, 0);
            mma_bf16(s[mt][nt], a0, qv.x, qv.y);
            mma_bf16(s[mt][nt], a1, qv.z, qv.w);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int kk = kg + 8 * (k >> 1);
            if (kk >= a.C || (a.causal && kk > qi[nt][k & 1])) s[mt][nt][k] = -INFINITY;
          }
      }
      float c[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = scale_log2;
      softmax_step<HD, NT>(s, c, 0.f, 1.f, acc);
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = s[mt][nt][2 * h], p1 = s[mt][nt][2 * h + 1];
            const uint32_t hi = pack_bf16(p0, p1);
            ph[nt][h] = transpose8x8(hi);
            pl[nt][h] = transpose8x8(pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u)));
          }
        }
        const __nv_bfloat16* vr[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int key = key0 + 16 * mt + 2 * t + (q & 1) + 8 * (q >> 1);
          vr[q] = key < a.C ? vn + (size_t)key * HD + g * NV : nullptr;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          uint32_t vw[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            vw[q] = vr[q] ? *reinterpret_cast<const uint32_t*>(vr[q] + 2 * i) : 0u;
            vn_top = __vmaxu2(vn_top, vw[q] & 0x7fff7fffu);
          }
          const uint32_t va[4] = {__byte_perm(vw[0], vw[1], 0x5410u), __byte_perm(vw[0], vw[1], 0x7632u),
                                  __byte_perm(vw[2], vw[3], 0x5410u), __byte_perm(vw[2], vw[3], 0x7632u)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16(acc.o[nt][i], va, ph[nt][0], ph[nt][1]);
            mma_bf16(acc.o[nt][i], va, pl[nt][0], pl[nt][1]);
          }
        }
      }
    }
    bool beyond = max(ve_top, top_exponent(max(vn_top & 0xffffu, vn_top >> 16))) > kKv8EmaxAttn;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) beyond |= kv8_far(acc.m[nt][0]) || kv8_far(acc.m[nt][1]);
    if (beyond) atomicExch(a.status, kStatusValue);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) acc.l[nt][e] += __shfl_xor_sync(0xffffffffu, acc.l[nt][e], o);

    // four columns (4 k .. of the lane group's NV) of row 2t + e
    auto out4 = [&](int nt, int e, int k) {
      return make_float4(acc.o[nt][2 * k][e], acc.o[nt][2 * k][2 + e], acc.o[nt][2 * k + 1][e], acc.o[nt][2 * k + 1][2 + e]);
    };
    if (a.cluster) {
      // every warp's output and (maximum, sum) to shared memory, the output to
      // its own ring; then the unit's threads merge, four columns of a row each, and
      // where a unit has several CTAs, the threads of all merge what these made
      float* mine = reinterpret_cast<float*>(ring);
      float2* ml = reinterpret_cast<float2*>(smem + R::oMl);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * t + e;
          if (g == 0) ml[warp * 32 + r] = make_float2(acc.m[nt][e], acc.l[nt][e]);
#pragma unroll
          for (int k = 0; k < NV / 4; ++k) *reinterpret_cast<float4*>(mine + r * HD + g * NV + 4 * k) = out4(nt, e, k);
        }
      }
      __syncthreads();
      float4* joined = reinterpret_cast<float4*>(smem + R::oJoin);
      float2* joined_ml = reinterpret_cast<float2*>(smem + R::oJoin + R::kJoin);
      const int items = *abort || p.b >= a.B ? 0 : a.prows * (HD / 4);
      if (a.group < W) {  // rolled: the usual calls' code stays short
        for (int i = threadIdx.x - 32 * lead; i < items; i += 32 * a.group) {
          const int r = i / (HD / 4), c4 = i % (HD / 4);
          if (row0 + r >= grp_rows) break;
          float M = -INFINITY;
#pragma unroll 1
          for (int k = lead; k < lead + a.group; ++k) M = fmaxf(M, ml[k * 32 + r].x);
          Kv8Sum<1> sum;
#pragma unroll 1
          for (int sl = 0; sl < min(kMergeSlices, a.group); ++sl) {
            Kv8Sum<1> s;
#pragma unroll 1
            for (int k = lead + sl; k < lead + a.group; k += kMergeSlices)
              s.add(ml[k * 32 + r], M, reinterpret_cast<const float4*>(smem + k * R::kWarp + (r * HD + 4 * c4) * 4), 0);
            sum.add(s);
          }
          sum.store(kv8_out_row(a, p.b, hk, row0 + r) + 4 * c4);
        }
        break;
      }
      for (int i = threadIdx.x; i < items; i += 32 * W) {
        const int r = i / (HD / 4), c4 = i % (HD / 4);
        if (row0 + r >= grp_rows) break;
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < W; ++k) M = fmaxf(M, ml[k * 32 + r].x);
        Kv8Sum<1> sum;
#pragma unroll
        for (int sl = 0; sl < kMergeSlices; ++sl) {  // the merge kernel's order of additions
          Kv8Sum<1> s;
#pragma unroll
          for (int k = sl; k < W; k += kMergeSlices)
            s.add(ml[k * 32 + r], M, reinterpret_cast<const float4*>(smem + k * R::kWarp + (r * HD + 4 * c4) * 4), 0);
          sum.add(s);
        }
        if (a.cluster == 1) {
          sum.store(kv8_out_row(a, p.b, hk, row0 + r) + 4 * c4);
        } else {
          joined[i] = sum.v[0];
          if (c4 == 0) joined_ml[r] = make_float2(M, sum.l);
        }
      }
      if (a.cluster == 1) break;
      __syncwarp();
      cluster_sync();
      for (int i = threadIdx.x * a.cluster + rank; i < items; i += 32 * W * a.cluster) {
        const int r = i / (HD / 4), c4 = i % (HD / 4);
        if (row0 + r >= grp_rows) break;
        float2 y[kMaxCluster];
        float4 x[kMaxCluster];
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          y[k] = make_float2(-INFINITY, 0.f);
          x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < a.cluster) {
            y[k] = ld_cluster_v2(cluster_addr(joined_ml + r, k));
            x[k] = ld_cluster_v4(cluster_addr(joined + i, k));
          }
        }
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) M = fmaxf(M, y[k].x);
        Kv8Sum<1> sum;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) sum.add(y[k], M, &x[k], 0);
        sum.store(kv8_out_row(a, p.b, hk, row0 + r) + 4 * c4);
      }
      __syncwarp();
      cluster_sync();  // no CTA leaves while a peer may still read its shared memory
      break;
    }
    if (!ok) break;
    const bool whole = t0 == 0 && t1 == p.nt;
    const size_t part = (size_t)worker * 2 + (t0 > 0 ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * t + e;
        if (row0 + r >= grp_rows) continue;
        const float l = acc.l[nt][e];
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.0f / l;
          uint2* dst = reinterpret_cast<uint2*>(kv8_out_row(a, p.b, hk, row0 + r) + g * NV);
#pragma unroll
          for (int k = 0; k < NV / 4; ++k) {
            const float4 v = out4(nt, e, k);
            dst[k] = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
          }
        } else {
#pragma unroll
          for (int k = 0; k < NV / 4; ++k) *kv8_part(a, part, (g * NV) / 4 + k, r) = out4(nt, e, k);
          if (g == 0) a.ml[part * a.prows + r] = make_float2(acc.m[nt][e], l);
        }
      }
    }
  }
  if (*abort) {  // copies in flight land before the CTA's shared memory goes
    const uint64_t start = globaltimer();
    while (globaltimer() - start < 2000000ull) __nanosleep(1000);
  }
}

// Merge of the parts.  A thread makes 4 N columns of an output row, a warp those
// of 32 consecutive rows (of fewer rows and more columns where a part has
// fewer), a CTA of 8 warps those of one unit.  Single tokens' units have some
// 50 parts of few rows: the eight warps share them (S = 8; one warp alone would
// wait for them round by round, 15 us for 4 sequences of 131072 rows).  The
// 256-row units of the tensor-core kernel have fewer parts and rows enough for
// a warp each (S = 1).  One warp works out where the shares' borders cut the
// unit (done by every warp it took longer than the parts: 16 us for 8 prompt
// pieces), all of them where there are many sequences (256: 28 us by one, 18 by
// all); a unit that one worker finished is already written, and one without
// any key (an empty sequence without new tokens) gets zeros.  What is read
// before pdl_wait, the lengths, no kernel of the call writes, and the
// attention kernel lets this one start only once it has itself waited for its
// predecessors; they are read past the first-level cache.
constexpr int kMergeWarps = 8;

template <int HD, int S, int N, int SUBS>
__global__ void __launch_bounds__(32 * kMergeWarps) kv8_merge_kernel(Kv8AttnArgs a, int ctas) {
  constexpr int CN = HD / (4 * N);
  __shared__ int costs[kMergeWarps][3], cut[3];
  __shared__ float top[kMergeWarps / S][S][32];
  __shared__ Kv8Sum<N> sums[kMergeWarps / S][S > 1 ? S : 1][S > 1 ? 32 : 1];
  const int lane = threadIdx.x % 32, slice = threadIdx.x / 32 % S, sub = threadIdx.x / (32 * S);
  const int grp_rows = a.Hq / a.Hkv * a.C;
  const unsigned all = blockIdx.x / (unsigned)ctas;  // `ctas` CTAs a unit
  const int b = (int)(all / a.units), unit = (int)(all - (unsigned)b * a.units);
  // Cost of the call, and of the sequences before b, by the first warp, or where
  // it would have to go round by all.
  const bool many = a.B > 32;
  if (many || threadIdx.x < 32) {
    int total = 0, before = 0, own = 0;
    for (int i = threadIdx.x; i < a.B; i += many ? 32 * kMergeWarps : 32) {
      const int nt = kv8_tiles(a, kv8_len(a, i)), cost = kv8_cost(a, nt) * a.units;
      total += cost;
      if (i < b) before += cost;
      if (i == b) own = nt;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    before = __reduce_add_sync(0xffffffffu, before);
    own = __reduce_add_sync(0xffffffffu, own);
    if (lane == 0) {
      costs[threadIdx.x / 32][0] = total;
      costs[threadIdx.x / 32][1] = before;
      costs[threadIdx.x / 32][2] = own;
    }
    if (many) __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; many && i < kMergeWarps; ++i) {
        total += costs[i][0];
        before += costs[i][1];
        own += costs[i][2];
      }
      const int share = max((total + a.workers - 1) / a.workers, 1);
      const int first = before + unit * (own + a.ovh) + a.ovh;  // the unit's first tile
      cut[0] = first / share;
      cut[1] = (first + max(own, 1) - 1) / share;
      cut[2] = own;
    }
  }
  const int item = ((int)(blockIdx.x - all * ctas) * (kMergeWarps / S) + sub) * 32 + lane;
  const int row_tiles = a.units / a.Hkv, hk = unit / row_tiles;
  const int cn = item / a.prows, rr = item - cn * a.prows, r = unit % row_tiles * a.rows + rr;
  const bool mine = cn < CN && r < grp_rows;
  __syncthreads();
  const int c0 = cut[0], n = cut[1] - c0, nt = cut[2];
  pdl_wait();
  if (nt > 0 && n == 0) return;  // uniform over the CTA
  // Part 0 (with its sub-parts) is the unit's beginning, slot 1 of its worker; the
  // others are slots 0.  The slots' loads go out in groups, whole ones: what a
  // group lacks is read as an empty part, so that no remainder waits on its own.
  const size_t mstep = a.prows, pstep = mstep * (HD / 4);
  const float2* ml = a.ml + (size_t)c0 * 2 * SUBS * mstep + (mine ? rr : 0);
  const float4* src = kv8_part(a, (size_t)c0 * 2 * SUBS, mine ? cn * N : 0, mine ? rr : 0);
  const int last = nt > 0 ? n : -1;
  auto at = [](int i, int u) { return (size_t)(i * 2 * SUBS + (i == 0 ? SUBS : 0) + u); };
  constexpr int kGroup = 8 / SUBS;
  float M = -INFINITY;
#pragma unroll 1
  for (int i0 = slice; i0 <= last; i0 += kGroup * S) {
    float m[kGroup][SUBS];
#pragma unroll
    for (int k = 0; k < kGroup; ++k)
#pragma unroll
      for (int u = 0; u < SUBS; ++u) m[k][u] = i0 + k * S <= last ? ml[at(i0 + k * S, u) * mstep].x : -INFINITY;
#pragma unroll
    for (int k = 0; k < kGroup; ++k)
#pragma unroll
      for (int u = 0; u < SUBS; ++u) M = fmaxf(M, m[k][u]);
  }
  if constexpr (S > 1) {
    top[sub][slice][lane] = M;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < S; ++k) M = fmaxf(M, top[sub][k][lane]);
  }
  Kv8Sum<N> s;
  constexpr int kGroup2 = N * SUBS >= 4 ? 2 : 8 / (N * SUBS);
#pragma unroll 1
  for (int i0 = slice; i0 <= last; i0 += kGroup2 * S) {
    float2 m[kGroup2][SUBS];
    float4 x[kGroup2][SUBS][N];
#pragma unroll
    for (int k = 0; k < kGroup2; ++k) {
      const int i = i0 + k * S;
#pragma unroll
      for (int u = 0; u < SUBS; ++u) {
        m[k][u] = make_float2(-INFINITY, 0.f);
        if (i <= last) m[k][u] = ml[at(i, u) * mstep];
#pragma unroll
        for (int c = 0; c < N; ++c) {
          x[k][u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i <= last) x[k][u][c] = src[at(i, u) * pstep + c * mstep];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kGroup2; ++k)
#pragma unroll
      for (int u = 0; u < SUBS; ++u) s.add(m[k][u], M, x[k][u], 1);
  }
  if constexpr (S > 1) {
    sums[sub][slice][lane] = s;
    __syncthreads();
    if (slice != 0) return;
    s = Kv8Sum<N>();
#pragma unroll
    for (int k = 0; k < S; ++k) s.add(sums[sub][k][lane]);
  }
  if (mine) s.store(kv8_out_row(a, b, hk, r) + 4 * N * cn);
}

template <int HD, int NT>
cudaError_t run_mma(const Kv8AttnArgs& a, cudaStream_t st) {
  constexpr int W = kv8_mma_warps(HD, 8 * NT);
  using R = Ring<HD, W>;
  cudaError_t e = set_smem_once<kv8_attn_kernel<HD, NT, W>>(R::kSmem);
  if (e != cudaSuccess) return e;
  const uint64_t rows = (uint64_t)a.B * a.Hkv * a.cap;
  CUtensorMap mK, mV;
  if (!make_tmap_2d(&mK, a.K, HD, rows, HD, HD, kStep, true, HD) ||
      !make_tmap_2d(&mV, a.V, HD, rows, HD, HD, kStep, true, HD))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.cluster ? cdiv((int64_t)a.B * a.units, W / a.group) * a.cluster : kKv8Ctas);
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = R::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = kProgrammaticLaunch;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kv8_attn_kernel<HD, NT, W>, mK, mV, a, 1.4426950408889634f / sqrtf((float)HD));
}

template <int HD>
cudaError_t run_rows(const Kv8AttnArgs& a, cudaStream_t st) {
  if (a.rows == 8) return run_mma<HD, 1>(a, st);
  if (a.rows == 16) return run_mma<HD, 2>(a, st);
  if constexpr (HD < 128) return run_mma<HD, 4>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace

// As many rows as the registers hold: the codes are read and converted once for
// all of a unit's rows.
int kv8_mma_rows(int hd, int64_t R) { return R <= 8 ? 8 : R <= 16 || hd == 128 ? 16 : 32; }

cudaError_t launch_kv8_attention_mma(const Kv8AttnArgs& a, cudaStream_t st) {
  switch (a.hd) {
    case 32: return run_rows<32>(a, st);
    case 64: return run_rows<64>(a, st);
    case 128: return run_rows<128>(a, st);
  }
  return cudaErrorInvalidValue;
}

template <int HD, int S, int N, int SUBS = 1>
static cudaError_t run_merge(const Kv8AttnArgs& a, cudaStream_t st) {
  const int ctas = cdiv((int64_t)a.prows * (HD / (4 * N)), 32 * (kMergeWarps / S));
  return launch_pdl(kv8_merge_kernel<HD, S, N, SUBS>, dim3((unsigned)(a.B * a.units * ctas)), dim3(32 * kMergeWarps), 0, st, a,
                    ctas);
}

template <int HD>
static cudaError_t run_merge_rows(const Kv8AttnArgs& a, cudaStream_t st) {
  if (a.rows < 128) return run_merge<HD, kMergeSlices, 1>(a, st);
  // By the parts that a unit has (hd 128; 19 of them, a canvas over 131072 rows:
  // 124.1 us, against 140.1 with a warp for all parts and 126.5 with two; 9, over
  // 8192 rows: 29.9 with two, against 37.9 with one and 32.0 with four; 2, prompt
  // pieces: 40.7 with one, against 44.3 with two).
  const int64_t units = (int64_t)a.B * a.units;
  if (a.subs == 2) return a.workers >= 8 * units ? run_merge<HD, 8, 1, 2>(a, st) : run_merge<HD, 2, 2, 2>(a, st);
  if (a.workers >= 16 * units) return run_merge<HD, 4, 2>(a, st);
  return a.workers >= 4 * units ? run_merge<HD, 2, 2>(a, st) : run_merge<HD, 1, 4>(a, st);
}

cudaError_t launch_kv8_merge(const Kv8AttnArgs& a, cudaStream_t st) {
  switch (a.hd) {
    case 32: return run_merge<32, kMergeSlices, 1>(a, st);
    case 64: return run_merge_rows<64>(a, st);
    case 128: return run_merge_rows<128>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dg

// Matrices of 4-bit weights with a scale per group, times a few rows.
//
//   y[m][n] = coef alpha[m] sum_k x[m][k] s[n][k / group] (c[n][k] - 8) + resid[m][n]
//
// The weights' bytes bound it (2 M flops a weight, 32 rows at most), so the
// codes lie in memory as the tensor cores take them: a tile of 16 rows by 64
// columns is 512 consecutive bytes, 16 for each lane of the warp that multiplies
// it, and the tiles of 64 rows lie side by side: [N / 64][K / 64][4 tiles][32
// lanes][16 bytes].  Lane 4 g + t holds rows g and g + 8 of its tile at columns 32 p +
// 8 t + i, p = 0, 1, i = 0..7.  Word j of its four is the A operand of one m16n8k16
// product: of the columns i = 4 (j % 2) + 0..3 of half p = j / 2, nibble r + 2 u
// (+ 4) is row g + 8 r at column i = 4 (j % 2) + 2 u (+ 1).  The order of a
// product's inner index is free as long as both operands follow it, so x is read
// in 16-byte pieces of a row.  Scales: bf16, [N / 64][K / group][8 g][4 tiles][rows g
// and g + 8], 16 bytes for a lane.
#include <cfloat>
#include <climits>
#include <type_traits>

#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kW4Rows = 16, kW4Cols = 64;  // a tile
constexpr int kW4Tiles = 4;                // tiles side by side
constexpr int kW4Bytes = kW4Rows * kW4Cols / 2;
constexpr int kW4MaxM = 32;

// Tile (rt, kb) in the order of memory, and the place of a group's scales of the rows
// g, g + 8 of row tile rt (in pairs).
DG_DEV size_t w4_tile(int rt, int kb, int KB) { return ((size_t)(rt / kW4Tiles) * KB + kb) * kW4Tiles + rt % kW4Tiles; }
DG_DEV size_t w4_scale(int rt, int group, int KG, int g) {
  return (((size_t)(rt / kW4Tiles) * KG + group) * 8 + g) * kW4Tiles + rt % kW4Tiles;
}

// Column of the tile at which the lane's word j begins.
DG_DEV int w4_col(int j, int t) { return 32 * (j / 2) + 8 * t + 4 * (j % 2); }

DG_DEV uint32_t f32_to_bf16_bits(float f) { return pack_bf16(f, 0.f) & 0xffffu; }

// ---------------------------------------------------- quantise, pack, read --
struct W4StoreArgs {
  const void* W;       // bf16 [N][ld], or codes uint8 [N][ld]
  const uint16_t* s;   // codes' scales [N][K / group]
  uint32_t* codes;
  uint32_t* scales;    // a pair of bf16 each
  int* status;
  int N, K, group;
  int64_t ld;
};

// A warp writes the tiles of one group of columns (two tiles where the group is
// 128): rows rt * 16 ...  A matrix is laid out once, so this is the simplest form: loads of
// one element, and quantising reads the matrix twice (262144 x 2816: quantising 1.32 ms,
// given codes 0.66, reading back 0.62).
constexpr int kStoreWarps = 8;

template <bool kQuantize>
__global__ void __launch_bounds__(kStoreWarps * 32) w4_store_kernel(W4StoreArgs a) {
  pdl_wait();
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int KB = a.K / kW4Cols, span = a.group > kW4Cols ? 2 : 1, spans = KB / span;
  const int64_t id = (int64_t)blockIdx.x * kStoreWarps + threadIdx.x / 32;
  const int rt = (int)(id / spans), kb0 = (int)(id % spans) * span;
  if (rt >= (a.N + kW4Rows * kW4Tiles - 1) / (kW4Rows * kW4Tiles) * kW4Tiles) return;
  for (int half = 0; half < (a.group < kW4Cols ? 2 : 1); ++half) {
    // the group's columns: both halves of its tiles, or with groups of 32 one half
    const int p0 = a.group < kW4Cols ? half : 0, p1 = a.group < kW4Cols ? half + 1 : 2;
    uint32_t sc[2];
    if (kQuantize) {
      const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.W);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int n = rt * kW4Rows + g + 8 * r;
        float top = 0.f;
        bool bad = false;
        if (n < a.N)
          for (int kb = kb0; kb < kb0 + span; ++kb)
            for (int p = p0; p < p1; ++p)
              for (int i = 0; i < 8; ++i) {
                const float v = fabsf(__bfloat162float(W[(size_t)n * a.ld + kb * kW4Cols + 32 * p + 8 * t + i]));
                if (v <= FLT_MAX) top = fmaxf(top, v);
                else bad = true;
              }
        if (bad) atomicExch(a.status, kStatusValue);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        sc[r] = f32_to_bf16_bits(top / 7.0f);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int n = rt * kW4Rows + g + 8 * r;
        sc[r] = n < a.N ? a.s[(size_t)n * (a.K / a.group) + (kb0 * kW4Cols + 32 * p0) / a.group] : 0u;
      }
    }
    if (t == 0)
      a.scales[w4_scale(rt, (kb0 * kW4Cols + 32 * p0) / a.group, a.K / a.group, g)] = sc[0] | (sc[1] << 16);
    for (int kb = kb0; kb < kb0 + span; ++kb)
      for (int j = 2 * p0; j < 2 * p1; ++j) {
        uint32_t word = 0;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int n = rt * kW4Rows + g + 8 * r;
          const float s = __uint_as_float(sc[r] << 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t c = 8;
            if (n < a.N) {
              const size_t at = (size_t)n * a.ld + kb * kW4Cols + w4_col(j, t) + i;
              if (kQuantize) {
                const float v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.W)[at]);
                // a group of zeros has scale 0; NaN is stored as zero
                const float q = s > 0.f && v == v ? fminf(fmaxf(rintf(v / s), -7.f), 7.f) : 0.f;
                c = (uint32_t)((int)q + 8);
              } else {
                c = static_cast<const uint8_t*>(a.W)[at] & 15u;
              }
            }
            word |= c << (4 * (r + 2 * (i / 2) + 4 * (i % 2)));
          }
        }
        a.codes[(w4_tile(rt, kb, KB) * 32 + lane) * 4 + j] = word;
      }
  }
}

struct W4ReadArgs {
  const uint32_t* codes;
  const uint32_t* scales;
  float* out;
  int N, K, group;
  int64_t ld;
};

__global__ void __launch_bounds__(256) w4_read_kernel(W4ReadArgs a) {
  pdl_wait();
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;  // one word: two rows, four columns
  const int j = (int)(id % 4), lane = (int)(id / 4 % 32), g = lane / 4, t = lane % 4;
  const int64_t tile = id / 128;
  const int KB = a.K / kW4Cols, kb = (int)(tile / kW4Tiles % KB);
  const int rt = (int)(tile / kW4Tiles / KB) * kW4Tiles + (int)(tile % kW4Tiles);
  if (rt >= (a.N + kW4Rows - 1) / kW4Rows) return;
  const uint32_t word = a.codes[id];
  const int k = kb * kW4Cols + w4_col(j, t);
  const uint32_t sc = a.scales[w4_scale(rt, k / a.group, a.K / a.group, g)];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int n = rt * kW4Rows + g + 8 * r;
    if (n >= a.N) continue;
    const float s = __uint_as_float(r ? sc & 0xffff0000u : sc << 16);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = s * (float)((int)((word >> (4 * (r + 2 * (i / 2) + 4 * (i % 2)))) & 15u) - 8);
    float* dst = a.out + (size_t)n * a.ld + k;
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = v[i];
  }
}

// ---------------------------------------------------------------- products --
struct W4Args {
  const uint4* codes;
  const uint32_t* scales;
  const __nv_bfloat16* x;
  const float* alpha;          // [M] or null
  const __nv_bfloat16* resid;  // [M][ldr] or null
  void* y;                     // [M][ldy]
  float coef;
  int N, K, group, M;
  int64_t ldx, ldr, ldy;
  int f32;
  int wk;                      // warps that share a row tile's columns
};

constexpr int kW4Warps = 8;
constexpr int kW4Stages = 4;

DG_DEV void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
DG_DEV void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Warps that share a unit: as few as leave the waves of sets on an SM's `ctas`
// CTAs within 5 % of full (fewer barriers), all eight otherwise (one row, K = 2816,
// codes from HBM: 2816 rows with 8, 4, 2, 1 warps 4.6, 7.9, 14.7, 19.6 us; 9728 rows 6.4,
// 10.0, 16.8, 26.9; 262144 rows 78.3, 75.7, 72.6, 77.7, of which it takes 4).  It does
// not see that few columns leave warps without any: 262144 x 64 with 8, which it
// takes, 4, 2, 1 warps 17.7, 14.0, 13.2, 6.2 us, x 256 20.2, 17.9, 17.5, 12.3.
int w4_split(int units, int KB, int ctas) {
  for (int wk = 1; wk < kW4Warps && wk < KB; wk *= 2) {
    const int sets = cdiv(units, kW4Warps / wk), slots = ctas * kTargetCtas;
    if (cdiv(sets, slots) * slots <= sets * 1.05) return wk;
  }
  return kW4Warps;
}

// Four codes' pairs as bf16: the nibble in the low bits of 128 (the mantissa's
// unit there is 1), less 136.  Both are exact.
DG_DEV uint32_t w4_pair(uint32_t word, int i) {
  uint32_t v;  // (word >> 4 i) & mask | 128's bits, in one operation after the shift
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(word >> (4 * i)), "r"(0x000f000fu), "r"(0x43004300u));
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __nv_bfloat162(136.f, 136.f));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// D = A B, the sum's first product
DG_DEV void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

DG_DEV void w4_store(const W4Args& a, int m, int col, float v) {
  if (m >= a.M || col >= a.N) return;
  v *= a.alpha ? a.coef * a.alpha[m] : a.coef;
  if (a.resid) v += __bfloat162float(a.resid[m * a.ldr + col]);
  if (a.f32) static_cast<float*>(a.y)[m * a.ldy + col] = v;
  else static_cast<__nv_bfloat16*>(a.y)[m * a.ldy + col] = __float2bfloat16_rn(v);
}

// D += A B
DG_DEV void mma_bf16_more(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A unit is R row tiles and all their columns, shared by wk warps (every wk-th
// tile of 64 columns each); a CTA works on kW4Warps / wk units at a time, a set.  A
// warp's codes and scales come through a ring of cp.async copies that runs on over
// the borders of its units; a lane reads only what it copied itself, so it waits for
// nothing but its own copies.  Bound by latency for short matrices (4096 x 2816, one
// row: 3.9 us), by HBM for long ones (262144 x 2816: 76 us, 5.2 TB/s, 160
// instructions of a warp for 2048 codes).
template <int NT, int R, int SG>
__global__ void __launch_bounds__(kW4Warps * 32, 2) w4_matvec_kernel(W4Args a) {
  constexpr int S = kW4Stages, kStage = R * kW4Bytes + SG * 32 * 4 * R;  // a lane's scales: 4 bytes to a tile
  constexpr int kSteps = R == kW4Tiles ? 2 : 1;  // tiles of columns at a time: eight rows over 262144 x 2816 95 -> 88 us; short matrices lose 5 %
  extern __shared__ __align__(16) char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  char* ring = smem + warp * S * kStage;
  float* part = reinterpret_cast<float*>(smem + kW4Warps * S * kStage);  // [2][warps][R * NT * 4][32]
  const int KB = a.K / kW4Cols, KG = a.K / a.group, tiles = (a.N + kW4Rows - 1) / kW4Rows;
  const int wk = a.wk, per = kW4Warps / wk, sub = warp % wk;
  const int sets = (tiles + per * R - 1) / (per * R);
  const int sg_shift = a.group == 2 * kW4Cols ? 1 : 0;  // tiles that share a group

  int pset = blockIdx.x, pkb = sub, pslot = 0;  // what is copied next, and where it lies
  bool more = sub < KB;                         // (else no columns for this warp)
  const char *pc = nullptr, *ps = nullptr;
  auto seek = [&]() {
    const int rt0 = (pset * per + warp / wk) * R;
    more = more && pset < sets && rt0 < tiles;
    pc = reinterpret_cast<const char*>(a.codes) + w4_tile(rt0, sub, KB) * kW4Bytes + lane * 16;
    ps = reinterpret_cast<const char*>(a.scales + w4_scale(rt0, 0, KG, g));
  };
  auto issue = [&]() {
    if (more) {
      char* slot = ring + pslot;
#pragma unroll
      for (int r = 0; r < R; ++r) cp_async16(slot + r * kW4Bytes + lane * 16, pc + r * kW4Bytes);
#pragma unroll
      for (int q = 0; q < SG; ++q) {
        const char* s = ps + ((pkb * SG >> sg_shift) + q) * 128;
        if (R == kW4Tiles) cp_async16(slot + R * kW4Bytes + q * 512 + lane * 16, s);
        else cp_async4(slot + R * kW4Bytes + q * 128 + lane * 4, s);
      }
      pkb += wk;
      pc += wk * kW4Tiles * kW4Bytes;
      if (pkb >= KB) {
        pkb = sub;
        pset += gridDim.x;
        seek();
      }
    }
    cp_async_commit();
    pslot = pslot + kStage == S * kStage ? 0 : pslot + kStage;
  };
  seek();
  pdl_wait();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();

  // columns past the last row of x repeat it: their sums are not stored
  const __nv_bfloat16* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xp[n] = a.x + min(8 * n + g, a.M - 1) * a.ldx + 8 * t;
  int slot_at = 0, buf = 0;
  for (int set = blockIdx.x; set < sets; set += gridDim.x) {
    float y[R][NT][4] = {};
#pragma unroll kSteps
    for (int kb = sub; kb < KB; kb += wk) {
      uint4 b[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) b[n][p] = __ldg(reinterpret_cast<const uint4*>(xp[n] + kb * kW4Cols + 32 * p));
      issue();
      cp_async_wait<S - 1>();
      const char* slot = ring + slot_at;
      slot_at = slot_at + kStage == S * kStage ? 0 : slot_at + kStage;
      uint32_t sw[SG][R];
#pragma unroll
      for (int q = 0; q < SG; ++q) {
        const char* from = slot + R * kW4Bytes + q * 128 * R + lane * 4 * R;
        if (R == kW4Tiles) *reinterpret_cast<uint4*>(sw[q]) = *reinterpret_cast<const uint4*>(from);
        else sw[q][0] = *reinterpret_cast<const uint32_t*>(from);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4 cw = *reinterpret_cast<const uint4*>(slot + r * kW4Bytes + lane * 16);
        const uint32_t words[4] = {cw.x, cw.y, cw.z, cw.w};
        float acc[NT][4];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t A[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) A[i] = w4_pair(words[2 * p + h], i);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t b0 = h ? b[n][p].z : b[n][p].x, b1 = h ? b[n][p].w : b[n][p].y;
              if (h == 0 && (SG == 2 || p == 0)) mma_bf16_first(acc[n], A, b0, b1);
              else mma_bf16_more(acc[n], A, b0, b1);
            }
          }
          if (SG == 2 || p == 1) {
            const uint32_t s = sw[SG == 2 ? p : 0][r];
            const float s0 = __uint_as_float(s << 16), s1 = __uint_as_float(s & 0xffff0000u);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              y[r][n][0] += s0 * acc[n][0];
              y[r][n][1] += s0 * acc[n][1];
              y[r][n][2] += s1 * acc[n][2];
              y[r][n][3] += s1 * acc[n][3];
            }
          }
        }
      }
    }
    const int rt0 = (set * per + warp / wk) * R;
    auto store = [&](int r, int i, float v) {
      w4_store(a, 8 * (i / 4) + 2 * t + i % 2, (rt0 + r) * kW4Rows + g + 8 * (i % 4 / 2), v);
    };
    if (wk > 1) {
      // the warps' sums, in order, each warp some of the unit's values; the other half
      // of `part` is free at the next unit's barrier
      float* unit = part + (buf * kW4Warps + warp - sub) * R * NT * 128 + lane;
#pragma unroll
      for (int i = 0; i < R * NT * 4; ++i) unit[(sub * R * NT * 4 + i) * 32] = y[i / (NT * 4)][i / 4 % NT][i % 4];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / wk), "r"(wk * 32) : "memory");
      buf ^= 1;
      for (int i = sub; i < R * NT * 4; i += wk) {
        float v = 0.f;
        for (int w = 0; w < wk; ++w) v += unit[(w * R * NT * 4 + i) * 32];
        store(i / (NT * 4), i % (NT * 4), v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R * NT * 4; ++i) store(i / (NT * 4), i % (NT * 4), y[i / (NT * 4)][i / 4 % NT][i % 4]);
    }
  }
  cp_async_wait<0>();
}

template <int NT, int R, int SG>
cudaError_t launch_w4(const W4Args& args, cudaStream_t st) {
  W4Args a = args;
  const int tiles = cdiv(a.N, kW4Rows), units = cdiv(tiles, R), KB = a.K / kW4Cols;
  constexpr int ctas = 2;
  a.wk = w4_split(units, KB, ctas);
  const int ring = kW4Warps * kW4Stages * R * (kW4Bytes + SG * 128);
  const int part = 2 * kW4Warps * R * NT * 128 * (int)sizeof(float);
  const cudaError_t e = set_smem_once<w4_matvec_kernel<NT, R, SG>>(ring + part);
  if (e != cudaSuccess) return e;
  const int sets = cdiv(units, kW4Warps / a.wk);
  return launch_pdl(w4_matvec_kernel<NT, R, SG>, dim3(sets < ctas * kTargetCtas ? sets : ctas * kTargetCtas), dim3(kW4Warps * 32),
                    (size_t)(ring + (a.wk > 1 ? part : 0)), st, a);
}

// More than eight rows over many row tiles: x no longer stays in L1 beside the rings
// (it would come from L2 twice as often as the codes from HBM), so all warps of a CTA
// work on the same columns at the same time, on row tiles of their own, and x lies in
// shared memory for kW4Chunk tiles of columns at a time, in the order of the products'
// operands (32 rows over 262144 x 2816: 167 us, 203 MB of codes and scales in 89 us at
// 131072; the MMAs alone are 8 cycles each of a quarter SM, 79 us of it).  A warp has a pair of neighbouring row tiles, whose codes of a tile of
// columns are one piece of memory: one lane copies a chunk's (cp.async.bulk, two chunks
// to a warp), so that little but the codes' own work is left to the others.  A CTA has
// an equal share of all pairs, 16 at a time; a rest of eight or fewer goes tile by tile.
constexpr int kW4WideWarps = 16;
constexpr int kW4Chunk = 4;

__device__ int g_w4_status;

DG_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// y += s a for two sums at once
DG_DEV void fma_two(float& y0, float& y1, float s, float a0, float a1) {
  asm("{\n .reg .b64 y, s, a;\n mov.b64 y, {%0, %1};\n mov.b64 s, {%2, %2};\n mov.b64 a, {%3, %4};\n"
      " fma.rn.f32x2 y, s, a, y;\n mov.b64 {%0, %1}, y;\n}\n"
      : "+f"(y0), "+f"(y1)
      : "f"(s), "f"(a0), "f"(a1));
}

template <int NT, int SG>
struct W4Wide {
  static constexpr int kX = NT * 1024;  // x of a tile of columns
  static constexpr int kCodes = kW4Chunk * 2 * kW4Bytes, kSlot = kCodes + kW4Chunk * SG * 128;
  static constexpr int kSmem = kW4WideWarps * 2 * kSlot + 2 * kW4Chunk * kX;
};

template <int NT, int SG>
__global__ void __launch_bounds__(kW4WideWarps * 32, 1) w4_wide_kernel(W4Args a) {
  using L = W4Wide<NT, SG>;
  extern __shared__ __align__(128) char smem[];
  __shared__ uint64_t full[kW4WideWarps][2];
  __shared__ int gave_up;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  char* ring = smem + warp * 2 * L::kSlot;
  char* xs = smem + kW4WideWarps * 2 * L::kSlot;  // [2][kW4Chunk][NT][2 halves][32 lanes][16 bytes]
  const int KB = a.K / kW4Cols, KG = a.K / a.group, chunks = (KB + kW4Chunk - 1) / kW4Chunk;
  const int sg_shift = a.group == 2 * kW4Cols ? 1 : 0;  // tiles of columns that share a group
  const int pairs = (a.N + 2 * kW4Rows - 1) / (2 * kW4Rows);
  const int p0 = (int)((int64_t)pairs * blockIdx.x / gridDim.x), p1 = (int)((int64_t)pairs * (blockIdx.x + 1) / gridDim.x);
  const int whole = (p1 - p0) / kW4WideWarps, rest = (p1 - p0) % kW4WideWarps, passes = whole + (rest > 0);
  // the first row tile of a pass, and how many
  auto tile_of = [&](int pass, int& n) {
    const int p = p0 + pass * kW4WideWarps;
    if (pass == whole && 2 * rest <= kW4WideWarps) {
      n = warp < 2 * rest ? 1 : 0;
      return 2 * p + warp;
    }
    n = pass < whole || warp < rest ? 2 : 0;
    return 2 * (p + warp);
  };

  if (tid == 0) {
    for (int i = 0; i < 2 * kW4WideWarps; ++i) mbar_init(&full[i / 2][i % 2], 1);
    gave_up = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();

  bool ok = true;
  int ppass = 0, pchunk = 0, pslot = 0;  // what is copied next, and where it lies
  auto issue = [&]() {
    if (ppass >= passes) return;
    int n;
    const int rt = tile_of(ppass, n);
    if (lane == 0 && n > 0 && ok) {
      const int kb = pchunk * kW4Chunk, nk = min(kW4Chunk, KB - kb);
      const int g0 = SG == 2 ? 2 * kb : kb >> sg_shift, ng = SG == 2 ? 2 * nk : nk >> sg_shift;
      uint64_t* bar = &full[warp][pslot];
      const uint32_t slot = smem_u32(ring) + pslot * L::kSlot;
      mbar_arrive_expect_tx(bar, nk * n * kW4Bytes + ng * 128);
      const char* codes = reinterpret_cast<const char*>(a.codes) + w4_tile(rt, kb, KB) * kW4Bytes;
      for (int k = 0; k < nk; ++k)
        bulk_load(slot + k * 2 * kW4Bytes, codes + k * kW4Tiles * kW4Bytes, n * kW4Bytes, bar);
      bulk_load(slot + L::kCodes, a.scales + w4_scale(rt / kW4Tiles * kW4Tiles, g0, KG, 0), ng * 128, bar);
    }
    pslot ^= 1;
    if (++pchunk == chunks) {
      pchunk = 0;
      ++ppass;
    }
  };
  // x of a chunk, 16 bytes (a lane's of one operand) at a time; rows past the last one
  // repeat it: their sums are not stored
  auto load_x = [&](int chunk, int buf) {
    const int kb = chunk * kW4Chunk, n = min(kW4Chunk, KB - kb) * NT * 64;
    for (int i = tid; i < n; i += kW4WideWarps * 32) {
      const int l = i % 32, p = i / 32 % 2, nt = i / 64 % NT, k = i / (64 * NT);
      const int m = min(8 * nt + l / 4, a.M - 1);
      cp_async16(xs + buf * kW4Chunk * L::kX + i * 16, a.x + m * a.ldx + (kb + k) * kW4Cols + 32 * p + 8 * (l % 4));
    }
    cp_async_commit();
  };
  load_x(0, 0);
  issue();
  issue();
  unsigned it = 0;  // chunks gone through
  auto next_x = [&](int pass, int chunk) {
    cp_async_wait<0>();
    __syncthreads();  // this chunk's x is there, and the one before is done with
    if (chunk + 1 < chunks) load_x(chunk + 1, (it + 1) & 1);
    else if (pass + 1 < passes) load_x(0, (it + 1) & 1);
  };
  auto go = [&](auto tiles, int pass, int rt) {
    constexpr int R = decltype(tiles)::value;
    float y[R][NT][4] = {};
    const int at_scale = L::kCodes + g * 16 + rt % kW4Tiles * 4;
#pragma unroll 1
    for (int chunk = 0; chunk < chunks; ++chunk) {
      next_x(pass, chunk);
      ok &= mbar_wait_warp(&full[warp][it & 1], it >> 1 & 1, &g_w4_status, &gave_up);
      const char* slot = ring + (it & 1) * L::kSlot;
      const uint4* xb = reinterpret_cast<const uint4*>(xs + (it & 1) * kW4Chunk * L::kX) + lane;
      const int nk = min(kW4Chunk, KB - chunk * kW4Chunk);
#pragma unroll
      for (int k = 0; k < kW4Chunk; ++k) {
        if (k >= nk) break;
        uint4 cw[R];
#pragma unroll
        for (int r = 0; r < R; ++r) cw[r] = *reinterpret_cast<const uint4*>(slot + (k * 2 + r) * kW4Bytes + lane * 16);
        float acc[R][NT][4];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint4 b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) b[n] = xb[k * NT * 64 + (n * 2 + p) * 32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t A[R][4];  // of all row tiles first: their products are independent
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const uint32_t word = p ? (h ? cw[r].w : cw[r].z) : (h ? cw[r].y : cw[r].x);
#pragma unroll
              for (int i = 0; i < 4; ++i) A[r][i] = w4_pair(word, i);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t b0 = h ? b[n].z : b[n].x, b1 = h ? b[n].w : b[n].y;
#pragma unroll
              for (int r = 0; r < R; ++r) {
                if (h == 0 && (SG == 2 || p == 0)) mma_bf16_first(acc[r][n], A[r], b0, b1);
                else mma_bf16_more(acc[r][n], A[r], b0, b1);
              }
            }
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (SG == 2 || p == 1) {
              const int group = SG == 2 ? 2 * k + p : k >> sg_shift;
              const uint32_t s = *reinterpret_cast<const uint32_t*>(slot + at_scale + group * 128 + r * 4);
              const float s0 = __uint_as_float(s << 16), s1 = __uint_as_float(s & 0xffff0000u);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                fma_two(y[r][n][0], y[r][n][1], s0, acc[r][n][0], acc[r][n][1]);
                fma_two(y[r][n][2], y[r][n][3], s1, acc[r][n][2], acc[r][n][3]);
              }
            }
          }
        }
      }
      __syncwarp();  // the slot is free
      issue();
      ++it;
    }
    if (!ok) return;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NT * 4; ++i) {
        const int m = 8 * (i / 4) + 2 * t + i % 2, col = (rt + r) * kW4Rows + g + 8 * (i % 4 / 2);
        w4_store(a, m, col, y[r][i / 4][i % 4]);
      }
  };
#pragma unroll 1
  for (int pass = 0; pass < passes; ++pass) {
    int n;
    const int rt = tile_of(pass, n);
    if (n == 2) {
      go(std::integral_constant<int, 2>{}, pass, rt);
    } else if (n == 1) {
      go(std::integral_constant<int, 1>{}, pass, rt);
    } else {
      for (int chunk = 0; chunk < chunks; ++chunk, ++it) next_x(pass, chunk);
    }
  }
  // after a wait that ran out no copies are begun; the ones on their way are given as long again
  if (!ok)
    for (const uint64_t t0 = globaltimer(); globaltimer() - t0 < kWaitLimitNs;) __nanosleep(1000);
}

template <int NT, int SG>
cudaError_t launch_w4_wide(const W4Args& a, cudaStream_t st) {
  using L = W4Wide<NT, SG>;
  const cudaError_t e = set_smem_once<w4_wide_kernel<NT, SG>>(L::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(w4_wide_kernel<NT, SG>, dim3(kTargetCtas), dim3(kW4WideWarps * 32), (size_t)L::kSmem, st, a);
}

// Four row tiles to a unit (x is read once for them, and their scales in one piece) where
// there are units enough for all SMs (K = 2816, one row, codes from HBM: 9728 rows 6.4 us
// against 7.7, 19456 rows 9.5 against 13.1, 38912 rows 14.3 against 19.3; 4864 rows 5.9
// against 4.9).  Above eight rows the kernel that keeps x in shared memory, from six
// pairs of row tiles to an SM on (32 rows of x: 29184 rows 26.8 us against 31.5, 19456
// rows 22.5 against 20.5; 16 rows: 19.1 against 20.9, 16.2 against 15.2).
template <int SG>
cudaError_t launch_w4_rows(const W4Args& a, cudaStream_t st) {
  const bool wide = cdiv(a.N, kW4Rows) >= (a.M <= 8 ? 4 : 12) * kTargetCtas;
  if (a.M <= 8) return wide ? launch_w4<1, kW4Tiles, SG>(a, st) : launch_w4<1, 1, SG>(a, st);
  if (a.M <= 16) return wide ? launch_w4_wide<2, SG>(a, st) : launch_w4<2, 1, SG>(a, st);
  return wide ? launch_w4_wide<4, SG>(a, st) : launch_w4<4, 1, SG>(a, st);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
dg_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DG_OK : DG_ERR_CUDA; }

dg_status check_w4_sizes(int32_t N, int32_t K, int32_t group) {
  if (N <= 0 || K <= 0 || group <= 0) return DG_ERR_ARG;
  if (group != 32 && group != 64 && group != 128) return DG_ERR_SHAPE;
  if (K % kW4Cols || K % group || K > 65536 || N > (1 << 24)) return DG_ERR_SHAPE;
  return DG_OK;
}

dg_status check_w4(const dg_w4* w) {
  if (!w || !w->codes || !w->scales) return DG_ERR_ARG;
  if (!aligned16(w->codes) || !aligned16(w->scales)) return DG_ERR_ARG;
  return check_w4_sizes(w->N, w->K, w->group);
}

template <bool kQuantize>
dg_status store(const dg_w4* w, const void* W, int64_t ld, const void* s, int32_t* status, void* stream) {
  W4StoreArgs a{W, static_cast<const uint16_t*>(s), static_cast<uint32_t*>(w->codes), static_cast<uint32_t*>(w->scales),
                status, w->N, w->K, w->group, ld};
  const int64_t spans = (int64_t)cdiv(w->N, kW4Rows * kW4Tiles) * kW4Tiles * (w->K / (w->group > kW4Cols ? w->group : kW4Cols));
  const int64_t ctas = (spans + kStoreWarps - 1) / kStoreWarps;
  if (ctas > INT_MAX) return DG_ERR_SHAPE;
  return from_cuda(launch_pdl(w4_store_kernel<kQuantize>, dim3((unsigned)ctas), dim3(kStoreWarps * 32), 0,
                              reinterpret_cast<cudaStream_t>(stream), a));
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" dg_status dg_w4_bytes(int32_t N, int32_t K, int32_t group, size_t* codes, size_t* scales) {
  if (!codes || !scales) return DG_ERR_ARG;
  dg_status e = check_w4_sizes(N, K, group);
  if (e) return e;
  const size_t rows = (size_t)cdiv(N, kW4Rows * kW4Tiles) * kW4Rows * kW4Tiles;
  *codes = rows * K / 2;
  *scales = rows * (K / group) * 2;
  return DG_OK;
}

extern "C" dg_status dg_w4_quantize(const dg_w4* w, const void* W, int64_t ldw, int32_t* status, void* stream) {
  dg_status e = check_w4(w);
  if (e) return e;
  if (!W || !status || ldw < w->K || reinterpret_cast<uintptr_t>(W) % 2 || reinterpret_cast<uintptr_t>(status) % 4)
    return DG_ERR_ARG;
  return store<true>(w, W, ldw, nullptr, status, stream);
}

extern "C" dg_status dg_w4_pack(const dg_w4* w, const void* codes, const void* scales, void* stream) {
  dg_status e = check_w4(w);
  if (e) return e;
  if (!codes || !scales || reinterpret_cast<uintptr_t>(scales) % 2) return DG_ERR_ARG;
  return store<false>(w, codes, w->K, scales, nullptr, stream);
}

extern "C" dg_status dg_w4_read(const dg_w4* w, float* out, int64_t ldo, void* stream) {
  dg_status e = check_w4(w);
  if (e) return e;
  if (!out || ldo < w->K || reinterpret_cast<uintptr_t>(out) % 4) return DG_ERR_ARG;
  W4ReadArgs a{static_cast<const uint32_t*>(w->codes), static_cast<const uint32_t*>(w->scales), out, w->N, w->K, w->group, ldo};
  const int64_t words = (int64_t)cdiv(w->N, kW4Rows * kW4Tiles) * kW4Tiles * (w->K / kW4Cols) * 128;
  if (words / 256 > INT_MAX - 1) return DG_ERR_SHAPE;
  return from_cuda(launch_pdl(w4_read_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0,
                              reinterpret_cast<cudaStream_t>(stream), a));
}

extern "C" dg_status dg_w4_matvec(const dg_w4* w, const void* x, int64_t ldx, int32_t M, const float* alpha, float coef,
                                  const void* resid, int64_t ldr, void* y, int64_t ldy, int32_t y_f32, void* stream) {
  dg_status e = check_w4(w);
  if (e) return e;
  if (!x || !y || M <= 0 || ldx < w->K || ldy < w->N || (resid && ldr < w->N)) return DG_ERR_ARG;
  if (!aligned16(x) || ldx % 8 || reinterpret_cast<uintptr_t>(y) % (y_f32 ? 4 : 2) ||
      reinterpret_cast<uintptr_t>(resid) % 2 || reinterpret_cast<uintptr_t>(alpha) % 4)
    return DG_ERR_ARG;
  if (M > kW4MaxM) return DG_ERR_SHAPE;
  W4Args a{static_cast<const uint4*>(w->codes), static_cast<const uint32_t*>(w->scales),
           static_cast<const __nv_bfloat16*>(x), alpha, static_cast<const __nv_bfloat16*>(resid), y, coef, w->N, w->K,
           w->group, M, ldx, ldr, ldy, y_f32 != 0, 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return from_cuda(w->group == 32 ? launch_w4_rows<2>(a, st) : launch_w4_rows<1>(a, st));
}

extern "C" dg_status dg_w4_status(int32_t* status, void* stream) {
  if (!status) return DG_ERR_ARG;
  void* word = nullptr;
  if (cudaGetSymbolAddress(&word, g_w4_status) != cudaSuccess) return DG_ERR_CUDA;
  return dg_read_status(word, status, stream);
}

// Shared declarations of the 8-bit prefix cache: its layout, the division of
// an attention call into pieces, and the launchers of its kernels.
#pragma once

#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {

constexpr int kKv8Block = 64;             // cached tokens per scale
constexpr int kKv8Bias = 127;             // exponent byte x: scale 2^(x - 127)
constexpr int kKv8Emin = -64, kKv8Emax = 118;
// Largest value scale attention takes.  A probability carries its block's value
// scale, p' = 2^(s + e - m + 8) with m the largest s + e; on blocks 2^104 below
// the largest scale it still has 2^30 above the smallest fp32, and the row's sum
// gets it back exactly; further down the sum would lose it.
constexpr int kKv8EmaxAttn = 40;
// Largest running maximum (log2 units; scores of 2^23).  A probability's argument is
// one rounding, s c + (ve - m): the rest of m's own rounding grows with m, up to
// 2 here, which the headroom below f16's largest holds.  Beyond, fp32 has not even
// the scores' units.
constexpr float kKv8Far = 16777216.0f;
constexpr int kKv8Ctas = kTargetCtas;     // CTAs of an attention launch (one per SM)
// Warps (workers) per CTA of the warp-MMA kernel for units of `rows` rows: as
// many as their registers allow.
constexpr int kv8_mma_warps(int hd, int rows) { return rows * hd <= 1024 ? 12 : 8; }
constexpr int kMaxCluster = 8;            // CTAs that finish a unit of a short cache together
constexpr int kStatusArg = 1, kStatusCapacity = 3;  // DG_ERR_ARG, DG_ERR_CAPACITY

// One attention call.  A unit is one row tile of one (sequence, kv head): the
// query rows of the group's heads, [B][Hkv][G C][hd] row-major as q lies in
// memory, cut into tiles of `rows`.  A unit's keys are cut into tiles of `tk`:
// first the cached rows, then (from a tile boundary on) the new ones.
struct Kv8AttnArgs {
  const void* q;             // bf16 [B][Hq][C][hd]
  const uint8_t *K, *V;      // codes [B][Hkv][cap][hd]
  const uint8_t *Ke, *Ve;    // exponent bytes [B][Hkv][nblk]
  const int* len;            // [B]
  const void *kn, *vn;       // bf16 [B][Hkv][C][hd] or null
  void* o;                   // bf16 [B*C][Hq*hd]
  float* part;               // fp32 [2 * workers * subs][hd / 4][prows][4]
  float2* ml;                // [2 * workers * subs][prows]: maximum (log2 units) and sum
  int* status;
  int B, C, Hq, Hkv, hd, cap, nblk;
  int causal;
  int rows, tk, units;       // rows per unit, keys per tile, units per sequence (Hkv * row tiles)
  int workers;               // warps or CTAs that the tiles are dealt to
  int subs;                  // parts of a piece: 2 where the tensor-core kernel's two row tiles share the rows
  int ovh;                   // what beginning a unit costs a worker, in tiles
  int prows;                 // rows of a part: min(rows, G C)
  int cluster;               // warp-MMA kernel: CTAs per unit, their warps' parts merged in shared memory (0: shares)
  int group;                 // then the warps of a CTA that share a unit: all, or with one CTA to a unit a divisor
};

// All work of a call, in the order (sequence, unit, tile), is dealt to the
// workers in equal contiguous shares, whatever the sequences' lengths: the
// device computes the division from the lengths, so the host never reads them
// and a captured graph follows a growing cache.  A unit counts its tiles and
// `ovh` more, for the queries, the pipeline's start and the output (without
// them workers with several short units ran twice as long as the others).  A
// unit cut by a share's border is left in parts, merged by the merge kernel: a
// worker's part that begins inside a unit goes to its slot 0 (there is one at
// most), the part of a unit that it begins and does not finish to its slot 1.
struct Kv8Piece {
  int b, len;                // sequence and its cached rows
  int nt, unit;              // tiles of each of its units; the unit
  int t0, t1;                // the piece's tiles (none where it ends before the unit's first)
  int cost;                  // share that the piece takes
};

DG_DEV int kv8_len(const Kv8AttnArgs& a, int b) {
  const int n = __ldcg(a.len + b);
  return min(max(n, 0), a.cap);
}
DG_DEV int kv8_tiles(const Kv8AttnArgs& a, int len) {
  return (len + a.tk - 1) / a.tk + (a.kn ? (a.C + a.tk - 1) / a.tk : 0);
}
// Four columns (4 c4 ..) of row r of a part: consecutive rows lie side by side,
// so that the kernels that hold a row in a thread write whole lines, and the
// merge reads a part from end to end.
DG_DEV float4* kv8_part(const Kv8AttnArgs& a, size_t slot, int c4, int r) {
  return reinterpret_cast<float4*>(a.part) + (slot * (a.hd / 4) + c4) * a.prows + r;
}
DG_DEV int kv8_cost(const Kv8AttnArgs& a, int nt) { return nt > 0 ? nt + a.ovh : 0; }
// What a warp knows of the call's division: the lengths of the first 32
// sequences, one in each lane (most calls have no more, and read them once).
struct Kv8Plan {
  int len;                   // of sequence `lane`
  int total, share;          // cost of the call (below 2^31 - 2^16 by the entry point's check), and of a worker
};
DG_DEV Kv8Plan kv8_plan(const Kv8AttnArgs& a) {
  const int lane = threadIdx.x & 31;
  Kv8Plan p;
  p.len = lane < a.B ? kv8_len(a, lane) : 0;
  int n = lane < a.B ? kv8_cost(a, kv8_tiles(a, p.len)) * a.units : 0;
  for (int b = lane + 32; b < a.B; b += 32) n += kv8_cost(a, kv8_tiles(a, kv8_len(a, b))) * a.units;
  p.total = __reduce_add_sync(0xffffffffu, n);
  p.share = max((p.total + a.workers - 1) / a.workers, 1);
  return p;
}
// The piece that begins at w in a share that ends at w1 (w < w1 <= the total; every
// lane of the calling warp gets the answer).  from: where the search begins, a
// sequence and the cost before it; zeros at first, then what the last call left
// there (375 sequences, 4 heads of 24 rows over up to 2000 rows: 275 us without
// it, 207 with).
DG_DEV Kv8Piece kv8_piece(const Kv8AttnArgs& a, const Kv8Plan& plan, int2& from, int w, int w1) {
  const int lane = threadIdx.x & 31;
  int base = from.y;
  Kv8Piece p{0, 0, 0, 0, 0, 0, w1 - w};
  for (int b0 = from.x; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    const int len = b0 == 0 ? plan.len : b < a.B ? kv8_len(a, b) : 0;
    const int nt = b < a.B ? kv8_tiles(a, len) : 0;
    const int mine = kv8_cost(a, nt) * a.units;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, w < base + incl);
    if (hit) {
      const int src = __ffs(hit) - 1;
      p.b = b0 + src;
      p.len = __shfl_sync(0xffffffffu, len, src);
      p.nt = __shfl_sync(0xffffffffu, nt, src);
      const int off = w - __shfl_sync(0xffffffffu, base + incl - mine, src), cost = p.nt + a.ovh;
      p.unit = off / cost;
      const int o0 = off - p.unit * cost, o1 = min(cost, o0 + (w1 - w));
      p.t0 = max(o0 - a.ovh, 0);
      p.t1 = max(o1 - a.ovh, 0);
      p.cost = o1 - o0;
      from = make_int2(b0, base);
      return p;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return p;
}

// Output row of query row r (< G C) of kv head g of sequence b.
DG_DEV __nv_bfloat16* kv8_out_row(const Kv8AttnArgs& a, int b, int g, int r) {
  const int h = g * (a.Hq / a.Hkv) + r / a.C, i = r % a.C;
  return reinterpret_cast<__nv_bfloat16*>(a.o) + (((size_t)b * a.C + i) * a.Hq + h) * a.hd;
}

// 16-byte chunk c of row r of a box of codes lies at chunk c ^ swz(r), the swizzle of
// the TMA copies over hd bytes: the fragment reads of eight lanes then fall
// into eight different bank groups (hd 128).
template <int HD>
DG_DEV int swz(int r) {
  return HD == 128 ? (r & 7) : HD == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
}

// Whether a running maximum lies too far from zero (none yet: no).
DG_DEV bool kv8_far(float m) { return fabsf(m) > kKv8Far && m != -INFINITY; }
// 2^e as a float, e clamped to the normal range.
DG_DEV float pow2i(int e) { return __uint_as_float((unsigned)(min(max(e, -126), 127) + 127) << 23); }
DG_DEV float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two E4M3 codes (low byte first) as two f16, exactly.
DG_DEV uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)codes));
  return r;
}
// Four codes as four f16: the low two in lo, the high two in hi.
DG_DEV void e4m3x4_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
// Two floats as E4M3 codes (low byte: lo), nearest even, saturating at 448.
DG_DEV uint32_t pack_e4m3(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

DG_DEV unsigned abs_top(const uint4& w) {
  return __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
}
// Smallest e with a largest magnitude <= 448 2^e, from its bf16 bits: 448 = 1.75 2^8.
DG_DEV int top_exponent(unsigned bits) {
  const int E = (int)(bits >> 7), m = (int)(bits & 127u);
  return E == 0 ? kKv8Emin : min(max(E - 127 - 8 + (m > 96 ? 1 : 0), kKv8Emin), kKv8Emax);
}

// Rows per unit of the warp-MMA kernel for R query rows per kv head.
int kv8_mma_rows(int hd, int64_t R);
// Parts i = s mod kMergeSlices of a unit are summed by slice s of the merge, the
// slices in order: one order of additions wherever the parts are merged.
constexpr int kMergeSlices = 8;

cudaError_t launch_kv8_attention_mma(const Kv8AttnArgs& a, cudaStream_t st);
cudaError_t launch_kv8_attention_tc(const Kv8AttnArgs& a, cudaStream_t st);
cudaError_t launch_kv8_merge(const Kv8AttnArgs& a, cudaStream_t st);

}  // namespace dg

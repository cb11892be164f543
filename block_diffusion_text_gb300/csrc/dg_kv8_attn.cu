// Attention over the 8-bit prefix cache for few query rows per kv head (single
// tokens, short canvases, head dims 32 and 64), and the merge of the parts.
//
// A warp is a worker: it streams its share of key tiles through a ring of its
// own in shared memory (cp.async, no barrier shared with other warps) and
// keeps queries, running maximum and sum, and the output of 16 MT rows in
// registers.  Work for single tokens is bound by the bytes of the cache, so
// what counts is loads in flight (24 KB a warp) and few instructions per code:
//  - The codes go from shared memory into the MMA fragments in one conversion
//    (two E4M3 to two f16, exact).  The fragments' index maps make that
//    possible: the sum over the head dim may run in any order, so lane t of a
//    quad owns the contiguous quarter t of a key row; the output columns may
//    be dealt in any order, so lane group g owns the contiguous eighth g of a
//    value row.
//  - Block scales never touch the codes.  The key scale joins the softmax
//    factor; the value scale 2^e joins the exponent of the probability,
//    p' = 2^(s + e - m), so that P' V sums codes, with m the running maximum of
//    s + e; the row sum takes p' 2^-e back.
//  - Queries enter as f16 scaled by a power of two per row (exact for elements
//    down to 2^-27 of the row's largest).  p' is rounded to f16 (2^-12 of its
//    value; 2^-33 of the largest at least, with the headroom of 2^8 below):
//    an eighth of the rounding of the bf16 output.
// New tokens' bf16 keys and values keep their exponent range: bf16 MMAs, P
// split into two bf16 parts (2^-17).
#include <cfloat>

#include "dg_kv8.cuh"

namespace dg {
namespace {

constexpr float kHeadroom = 8.0f;  // p' of a row's maximum is 2^8 ..
constexpr float kLazy = 4.0f;      // .. to 2^12: the maximum is followed when it grows by more than 2^4
constexpr int kStep = 32;          // keys per step

template <int HD>
struct Ring {
  static constexpr int kHalf = kStep * HD;     // codes of K (or V) of one step
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = HD == 128 ? 3 : HD == 64 ? 6 : 8;
  static constexpr int kWarp = kStages * kStage;
  static constexpr int oMl = kKv8Warps * kWarp;  // float2 [warps][32 rows]
  static constexpr int kSmem = oMl + kKv8Warps * 32 * 8;
};

// 16-byte chunk c of row r of a step lies at chunk c ^ swz(r): the fragment
// reads of eight lanes then fall into eight different bank groups (hd 128).
template <int HD>
DG_DEV int swz(int r) {
  return HD == 128 ? (r & 7) : HD == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
}

template <int HD, int MT>
struct Acc {
  float o[MT][HD / 8][4];
  float m[MT][2], l[MT][2];
};

// One step's scores to probabilities: s (raw products; rows g and g + 8 of
// each m-tile, keys nt * 8 + 2t, + 1) become p' = 2^(s c + ev - m + headroom).
template <int HD, int MT>
DG_DEV void softmax_step(float (&s)[MT][kStep / 8][4], const float (&c)[MT][2], float ev, float inv_ev,
                         Acc<HD, MT>& acc) {
  float mx[MT][2];
  bool need = false;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      float v = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < kStep / 8; ++nt) v = fmaxf(v, fmaxf(s[mt][nt][2 * hr], s[mt][nt][2 * hr + 1]));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
      mx[mt][hr] = fmaf(v, c[mt][hr], ev);
      need |= mx[mt][hr] > acc.m[mt][hr] + kLazy;
    }
  }
  if (__any_sync(0xffffffffu, need)) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const float mn = fmaxf(mx[mt][hr], acc.m[mt][hr]);
        const float corr = mn > acc.m[mt][hr] ? ex2_approx(acc.m[mt][hr] - mn) : 1.0f;
        acc.m[mt][hr] = mn;
        acc.l[mt][hr] *= corr;
#pragma unroll
        for (int n = 0; n < HD / 8; ++n) {
          acc.o[mt][n][2 * hr] *= corr;
          acc.o[mt][n][2 * hr + 1] *= corr;
        }
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      const float m = acc.m[mt][hr];
      const float off = ev - (m == -INFINITY ? 0.0f : m - kHeadroom);
      float sum = 0.f;
#pragma unroll
      for (int nt = 0; nt < kStep / 8; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = ex2_approx(fmaf(s[mt][nt][2 * hr + e], c[mt][hr], off));
          s[mt][nt][2 * hr + e] = p;
          sum += p;
        }
      }
      acc.l[mt][hr] = fmaf(sum, inv_ev, acc.l[mt][hr]);
    }
  }
}

// Words of the fragment slices: NB bytes from shared memory at p.
template <int NB>
DG_DEV void lds(uint32_t (&w)[NB / 4], const uint8_t* p) {
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

template <int HD, int MT>
__global__ void __launch_bounds__(32 * kKv8Warps, 1) kv8_attn_kernel(Kv8AttnArgs a, float scale_log2) {
  pdl_wait();
  pdl_trigger();  // the merge waits for this kernel's completion all the same
  using R = Ring<HD>;
  constexpr int SL = HD / 4;   // elements of a key row per quad lane
  constexpr int KS = HD / 16;  // k16 steps of Q K^T
  constexpr int NV = HD / 8;   // n-tiles of P V; columns per lane group
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  uint8_t* ring = smem + warp * R::kWarp;
  const int worker = warp * gridDim.x + blockIdx.x;  // consecutive shares on different SMs

  if (worker == 0) {
    for (int b = lane; b < a.B; b += 32)
      if (a.len[b] < 0 || a.len[b] > a.cap) atomicExch(a.status, kStatusCapacity);
  }
  int w = blockIdx.x, w1 = w + 1;  // local: the CTA's unit
  if (!a.local) {
    const int total = kv8_total(a), share = kv8_share(a, total);
    w1 = (int)min((long long)total, (worker + 1ll) * share);
    w = (int)min((long long)w1, (long long)worker * share);
  }
  const int grp_rows = a.Hq / a.Hkv * a.C, row_tiles = a.units / a.Hkv;

  while (w < w1) {
    Kv8Seq sq;
    int unit, t0, t1;
    if (a.local) {
      sq.b = w / a.units;
      sq.len = kv8_len(a, sq.b);
      sq.nt = kv8_tiles(a, sq.len);
      unit = w - sq.b * a.units;
      const int chunk = (sq.nt + kKv8Warps - 1) / kKv8Warps;
      t0 = min(warp * chunk, sq.nt);
      t1 = min(t0 + chunk, sq.nt);
    } else {
      sq = kv8_locate(a, w);
      unit = (w - sq.first) / sq.nt;
      t0 = w - sq.first - unit * sq.nt;
      t1 = min(sq.nt, t0 + (w1 - w));
    }
    const int hk = unit / row_tiles, row0 = unit % row_tiles * (16 * MT);
    const int ntc = (sq.len + kKv8Block - 1) / kKv8Block;
    const int tc1 = min(t1, ntc);  // cached tiles of the piece end here
    const size_t bh = (size_t)sq.b * a.Hkv + hk;
    const uint8_t* Kg = a.K + bh * a.cap * HD;
    const uint8_t* Vg = a.V + bh * a.cap * HD;
    const uint8_t* Ke = a.Ke + bh * a.nblk;
    const uint8_t* Ve = a.Ve + bh * a.nblk;
    const int nsteps = max(tc1 - t0, 0) * (kKv8Block / kStep);

    // Step i of the piece into its stage.  Rows past the sequence's end are
    // filled with zeros: what lies behind it never enters an MMA.
    auto issue = [&](int i) {
      if (i < nsteps) {
        const int key0 = t0 * kKv8Block + i * kStep;
        const int valid = sq.len - key0;
        uint8_t* dst = ring + (i % R::kStages) * R::kStage;
        constexpr int CPR = HD / 16;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint8_t* src = (kv ? Vg : Kg) + (size_t)key0 * HD;
#pragma unroll
          for (int p = 0; p < kStep * CPR / 32; ++p) {
            const int idx = p * 32 + lane, r = idx / CPR, c = idx % CPR;
            const bool there = r < valid;
            cp_async16(dst + kv * R::kHalf + r * HD + ((c ^ swz<HD>(r)) * 16), there ? src + r * HD + c * 16 : Kg,
                       there);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < R::kStages - 1; ++i) issue(i);

    // Queries: rows g and g + 8 of each m-tile, elements t SL + 4 j .. + 3.
    uint32_t qf[MT][KS][4];
    int qi[MT][2];    // position of the row's token among the new ones
    int qx[MT][2];
    const __nv_bfloat16* qrow[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const int r = row0 + mt * 16 + hr * 8 + g;
        const bool there = r < grp_rows;
        qi[mt][hr] = there ? r % a.C : 0;
        qrow[mt][hr] = there ? reinterpret_cast<const __nv_bfloat16*>(a.q) + (bh * grp_rows + r) * HD + t * SL : nullptr;
        uint2 raw[KS];
        unsigned top = 0;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          raw[j] = there ? *reinterpret_cast<const uint2*>(qrow[mt][hr] + 4 * j) : make_uint2(0, 0);
          top = __vmaxu2(top, __vmaxu2(raw[j].x & 0x7fff7fffu, raw[j].y & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int x = top < 128 ? 0 : max((int)(top >> 7) - 127 - 13, -100);
        qx[mt][hr] = x;
        const float f = pow2i(-x);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          qf[mt][j][hr] = pack_f16(__uint_as_float(raw[j].x << 16) * f, __uint_as_float(raw[j].x & 0xffff0000u) * f);
          qf[mt][j][2 + hr] = pack_f16(__uint_as_float(raw[j].y << 16) * f, __uint_as_float(raw[j].y & 0xffff0000u) * f);
        }
      }
    }
    Acc<HD, MT> acc;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        acc.m[mt][hr] = -INFINITY;
        acc.l[mt][hr] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc.o[mt][n][e] = 0.f;
    }

    int ke_next = 0, ve_next = 0, ke = 0, ve = 0;
    if (nsteps > 0) {
      ke_next = Ke[t0];
      ve_next = Ve[t0];
    }
#pragma unroll 1
    for (int i = 0; i < nsteps; ++i) {
      issue(i + R::kStages - 1);
      if (i % (kKv8Block / kStep) == 0) {
        ke = ke_next - kKv8Bias;
        ve = ve_next - kKv8Bias;
        const int nx = t0 + i / (kKv8Block / kStep) + 1;
        if (nx < tc1) {
          ke_next = Ke[nx];
          ve_next = Ve[nx];
        }
      }
      cp_async_wait<R::kStages - 1>();
      __syncwarp();
      const int valid = sq.len - (t0 * kKv8Block + i * kStep);
      if (valid > 0) {
        const uint8_t* sk = ring + (i % R::kStages) * R::kStage;
        const uint8_t* sv = sk + R::kHalf;
        float s[MT][kStep / 8][4];
#pragma unroll
        for (int nt = 0; nt < kStep / 8; ++nt) {
          const int r = nt * 8 + g;
          uint32_t kw[SL / 4];
          if constexpr (HD == 128) {
            uint32_t h0[4], h1[4];
            lds<16>(h0, sk + r * HD + (((2 * t) ^ swz<HD>(r)) * 16));
            lds<16>(h1, sk + r * HD + (((2 * t + 1) ^ swz<HD>(r)) * 16));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              kw[j] = h0[j];
              kw[4 + j] = h1[j];
            }
          } else if constexpr (HD == 64) {
            lds<16>(kw, sk + r * HD + ((t ^ swz<HD>(r)) * 16));
          } else {
            lds<8>(kw, sk + r * HD + (((t / 2) ^ swz<HD>(r)) * 16) + (t & 1) * 8);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            const uint32_t b0 = e4m3x2_f16x2(kw[j]), b1 = e4m3x2_f16x2(kw[j] >> 16);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma_f16_16816(s[mt][nt], qf[mt][j], b0, b1);
          }
        }
        if (valid < kStep) {
#pragma unroll
          for (int nt = 0; nt < kStep / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (nt * 8 + 2 * t + (e & 1) >= valid) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) s[mt][nt][e] = -INFINITY;
              }
        }
        float c[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hr = 0; hr < 2; ++hr) c[mt][hr] = scale_log2 * pow2i(qx[mt][hr] + ke);
        softmax_step<HD, MT>(s, c, (float)ve, pow2i(-ve), acc);
#pragma unroll
        for (int k2 = 0; k2 < kStep / 16; ++k2) {
          uint32_t pa[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            pa[mt][0] = pack_f16(s[mt][2 * k2][0], s[mt][2 * k2][1]);
            pa[mt][1] = pack_f16(s[mt][2 * k2][2], s[mt][2 * k2][3]);
            pa[mt][2] = pack_f16(s[mt][2 * k2 + 1][0], s[mt][2 * k2 + 1][1]);
            pa[mt][3] = pack_f16(s[mt][2 * k2 + 1][2], s[mt][2 * k2 + 1][3]);
          }
          uint32_t vw[4][NV / 4];  // rows 2t, 2t + 1, 2t + 8, 2t + 9; the lane group's columns
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 16 * k2 + 2 * t + (q & 1) + 8 * (q >> 1);
            if constexpr (HD == 128)
              lds<16>(vw[q], sv + r * HD + ((g ^ swz<HD>(r)) * 16));
            else if constexpr (HD == 64)
              lds<8>(vw[q], sv + r * HD + (((g / 2) ^ swz<HD>(r)) * 16) + (g & 1) * 8);
            else
              lds<4>(vw[q], sv + r * HD + (((g / 4) ^ swz<HD>(r)) * 16) + (g & 3) * 4);
          }
#pragma unroll
          for (int n = 0; n < NV; n += 2) {  // two n-tiles from one byte interleave of two rows
            const uint32_t sel = (n & 2) ? 0x7362u : 0x5140u;
            const uint32_t x0 = __byte_perm(vw[0][n / 4], vw[1][n / 4], sel);
            const uint32_t x1 = __byte_perm(vw[2][n / 4], vw[3][n / 4], sel);
            const uint32_t b00 = e4m3x2_f16x2(x0), b01 = e4m3x2_f16x2(x1);
            const uint32_t b10 = e4m3x2_f16x2(x0 >> 16), b11 = e4m3x2_f16x2(x1 >> 16);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_f16_16816(acc.o[mt][n], pa[mt], b00, b01);
              mma_f16_16816(acc.o[mt][n + 1], pa[mt], b10, b11);
            }
          }
        }
      }
      __syncwarp();  // the stage may be filled again
    }
    cp_async_wait<0>();

    // New tokens, in bf16, straight from global memory: a call has few of
    // them where this kernel is used.
    const __nv_bfloat16* kn = reinterpret_cast<const __nv_bfloat16*>(a.kn) + bh * a.C * HD;
    const __nv_bfloat16* vn = reinterpret_cast<const __nv_bfloat16*>(a.vn) + bh * a.C * HD;
#pragma unroll 1
    for (int key0 = (max(t0, ntc) - ntc) * kKv8Block, end = min((t1 - ntc) * kKv8Block, a.C); key0 < end;
         key0 += kStep) {
      float s[MT][kStep / 8][4];
#pragma unroll
      for (int nt = 0; nt < kStep / 8; ++nt) {
        const int key = key0 + nt * 8 + g;
        uint2 kw[KS];
#pragma unroll
        for (int j = 0; j < KS; j += 2) {
          const uint4 v = key < a.C ? *reinterpret_cast<const uint4*>(kn + (size_t)key * HD + t * SL + 4 * j)
                                    : make_uint4(0, 0, 0, 0);
          kw[j] = make_uint2(v.x, v.y);
          kw[j + 1] = make_uint2(v.z, v.w);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint2 r0 = make_uint2(0, 0), r1 = r0;
            if (qrow[mt][0]) r0 = *reinterpret_cast<const uint2*>(qrow[mt][0] + 4 * j);
            if (qrow[mt][1]) r1 = *reinterpret_cast<const uint2*>(qrow[mt][1] + 4 * j);
            const uint32_t qa[4] = {r0.x, r1.x, r0.y, r1.y};
            mma_bf16_16816(s[mt][nt], qa, kw[j].x, kw[j].y);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kk = key0 + nt * 8 + 2 * t + (e & 1);
            if (kk >= a.C || (a.causal && kk > qi[mt][e >> 1])) s[mt][nt][e] = -INFINITY;
          }
      }
      float c[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) c[mt][0] = c[mt][1] = scale_log2;
      softmax_step<HD, MT>(s, c, 0.f, 1.f, acc);
#pragma unroll
      for (int k2 = 0; k2 < kStep / 16; ++k2) {
        uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float p0 = s[mt][2 * k2 + (q >> 1)][2 * (q & 1)], p1 = s[mt][2 * k2 + (q >> 1)][2 * (q & 1) + 1];
            ph[mt][q] = pack_bf16(p0, p1);
            pl[mt][q] = pack_bf16(p0 - __uint_as_float(ph[mt][q] << 16),
                                  p1 - __uint_as_float(ph[mt][q] & 0xffff0000u));
          }
        }
        const __nv_bfloat16* vr[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int key = key0 + 16 * k2 + 2 * t + (q & 1) + 8 * (q >> 1);
          vr[q] = key < a.C ? vn + (size_t)key * HD + g * NV : nullptr;
        }
#pragma unroll
        for (int n = 0; n < NV; n += 2) {
          uint32_t vw[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) vw[q] = vr[q] ? *reinterpret_cast<const uint32_t*>(vr[q] + n) : 0u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t sel = e ? 0x7632u : 0x5410u;
            const uint32_t b0 = __byte_perm(vw[0], vw[1], sel), b1 = __byte_perm(vw[2], vw[3], sel);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_bf16_16816(acc.o[mt][n + e], ph[mt], b0, b1);
              mma_bf16_16816(acc.o[mt][n + e], pl[mt], b0, b1);
            }
          }
        }
      }
    }

    if (a.local) {
      // every warp's output and (maximum, sum) to its own ring, then all
      // threads merge: four columns of a row each
      float* mine = reinterpret_cast<float*>(ring);
      float2* ml = reinterpret_cast<float2*>(smem + R::oMl);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          float l = acc.l[mt][hr];
          l += __shfl_xor_sync(0xffffffffu, l, 1);
          l += __shfl_xor_sync(0xffffffffu, l, 2);
          const int r = mt * 16 + hr * 8 + g;
          if (t == 0) ml[warp * 32 + r] = make_float2(acc.m[mt][hr], l);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < NV; n += 4)
              *reinterpret_cast<float4*>(mine + r * HD + (2 * t + e) * NV + n) =
                  make_float4(acc.o[mt][n][2 * hr + e], acc.o[mt][n + 1][2 * hr + e], acc.o[mt][n + 2][2 * hr + e],
                              acc.o[mt][n + 3][2 * hr + e]);
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < a.prows * (HD / 4); i += 32 * kKv8Warps) {
        const int r = i / (HD / 4), c4 = i % (HD / 4);
        if (row0 + r >= grp_rows) break;
        float M = -INFINITY, L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kKv8Warps; ++k) M = fmaxf(M, ml[k * 32 + r].x);
#pragma unroll
        for (int k = 0; k < kKv8Warps; ++k) {
          const float2 p = ml[k * 32 + r];
          const float wk = p.x == -INFINITY ? 0.f : ex2_approx(p.x - M);
          const float4 x = *reinterpret_cast<const float4*>(smem + k * R::kWarp + (r * HD + 4 * c4) * 4);
          L = fmaf(wk, p.y, L);
          v.x = fmaf(wk, x.x, v.x);
          v.y = fmaf(wk, x.y, v.y);
          v.z = fmaf(wk, x.z, v.z);
          v.w = fmaf(wk, x.w, v.w);
        }
        const float inv = L == 0.f ? 0.f : 1.0f / L;
        *reinterpret_cast<uint2*>(kv8_out_row(a, sq.b, hk, row0 + r) + 4 * c4) =
            make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
      }
      return;
    }
    // Output, or a part of it: lane (g, t) holds columns 2 t NV .. + 2 NV of rows g and g + 8.
    const bool whole = t0 == 0 && t1 == sq.nt;
    const size_t slot = (size_t)worker * 2 + (t0 > 0 ? 0 : 1);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        float l = acc.l[mt][hr];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int r = mt * 16 + hr * 8 + g;
        if (row0 + r >= grp_rows) continue;
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.0f / l;
          uint32_t* dst = reinterpret_cast<uint32_t*>(kv8_out_row(a, sq.b, hk, row0 + r) + 2 * t * NV);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < NV; n += 2)
              dst[(e * NV + n) / 2] = pack_bf16(acc.o[mt][n][2 * hr + e] * inv, acc.o[mt][n + 1][2 * hr + e] * inv);
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < NV; n += 4)
              *kv8_part(a, slot, ((2 * t + e) * NV + n) / 4, r) =
                  make_float4(acc.o[mt][n][2 * hr + e], acc.o[mt][n + 1][2 * hr + e], acc.o[mt][n + 2][2 * hr + e],
                              acc.o[mt][n + 3][2 * hr + e]);
          if (t == 0) {
            const float m = acc.m[mt][hr];
            a.ml[slot * a.prows + r] = make_float2(m == -INFINITY ? m : m - kHeadroom, l);
          }
        }
      }
    }
    w += t1 - t0;
  }
}

// Merge of the parts.  A thread makes four columns of one output row, a warp 32
// consecutive float4 of a unit's parts; the shares' borders are recomputed, a
// unit that one worker finished is already written, and one without any key
// (an empty sequence without new tokens) gets zeros.  What it reads before
// pdl_wait, the lengths, no kernel of the call writes, and the attention
// kernel lets this one start only once it has itself waited for its
// predecessors; they are read past the first-level cache.
template <int HD>
__global__ void __launch_bounds__(256) kv8_merge_kernel(Kv8AttnArgs a) {
  constexpr int C4 = HD / 4;
  const int lane = threadIdx.x % 32;
  const int grp_rows = a.Hq / a.Hkv * a.C;
  const int per = (a.prows * C4 + 31) / 32;  // warps per unit
  const unsigned wid = blockIdx.x * 8 + threadIdx.x / 32, all = wid / per;
  const int b = (int)(all / a.units), unit = (int)(all - (unsigned)b * a.units);
  if (b >= a.B) return;
  const int item = (int)(wid - all * per) * 32 + lane;
  const int row_tiles = a.units / a.Hkv, hk = unit / row_tiles;
  const int c4 = item / a.prows, rr = item - c4 * a.prows, r = unit % row_tiles * a.rows + rr;
  const bool mine = c4 < C4 && r < grp_rows;
  const int nt = kv8_tiles(a, kv8_len(a, b));
  const int total = kv8_total(a), share = kv8_share(a, total);
  int first = 0;
  for (int i = lane; i < b; i += 32) first += kv8_tiles(a, kv8_len(a, i)) * a.units;
#pragma unroll
  for (int o = 16; o; o >>= 1) first += __shfl_xor_sync(0xffffffffu, first, o);
  first += unit * nt;
  const int c0 = first / share, c1 = (first + max(nt, 1) - 1) / share;
  pdl_wait();
  if (!mine || (nt > 0 && c0 == c1)) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = 0.f;
  if (nt > 0) {
    // part 0 is the unit's beginning (slot 1 of its worker), the others slots 0
    const float2* ml = a.ml + (size_t)c0 * 2 * a.prows + rr;
    const float4* src = kv8_part(a, (size_t)c0 * 2, c4, rr);
    const size_t mstep = 2 * (size_t)a.prows, pstep = mstep * C4;
    const float2 ml0 = ml[a.prows];
    const float4 v0 = src[(size_t)C4 * a.prows];
    const int n = c1 - c0;
    float M = ml0.x;
#pragma unroll 4
    for (int i = 1; i <= n; ++i) M = fmaxf(M, ml[i * mstep].x);
    const float w0 = ml0.x == -INFINITY ? 0.f : exp2f(ml0.x - M);
    L = w0 * ml0.y;
    acc = make_float4(v0.x * w0, v0.y * w0, v0.z * w0, v0.w * w0);
#pragma unroll 8
    for (int i = 1; i <= n; ++i) {
      const float2 p = ml[i * mstep];
      const float4 v = src[i * pstep];
      const float w = p.x == -INFINITY ? 0.f : exp2f(p.x - M);
      L = fmaf(w, p.y, L);
      acc.x = fmaf(v.x, w, acc.x);
      acc.y = fmaf(v.y, w, acc.y);
      acc.z = fmaf(v.z, w, acc.z);
      acc.w = fmaf(v.w, w, acc.w);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  *reinterpret_cast<uint2*>(kv8_out_row(a, b, hk, r) + 4 * c4) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

template <int HD, int MT>
cudaError_t run_mma(const Kv8AttnArgs& a, cudaStream_t st) {
  cudaError_t e = set_smem_once<kv8_attn_kernel<HD, MT>>(Ring<HD>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_attn_kernel<HD, MT>, dim3(a.local ? a.B * a.units : kKv8Ctas), dim3(32 * kKv8Warps), Ring<HD>::kSmem, st, a,
                    1.4426950408889634f / sqrtf((float)HD));
}

}  // namespace

// 16 rows, or 32 where the registers hold them and there are more than 16:
// the codes are then read and converted once for both row tiles.
int kv8_mma_rows(int hd, int64_t R) { return hd == 128 || R <= 16 ? 16 : 32; }

cudaError_t launch_kv8_attention_mma(const Kv8AttnArgs& a, cudaStream_t st) {
  switch (a.hd) {
    case 32: return a.rows == 16 ? run_mma<32, 1>(a, st) : run_mma<32, 2>(a, st);
    case 64: return a.rows == 16 ? run_mma<64, 1>(a, st) : run_mma<64, 2>(a, st);
    case 128: return run_mma<128, 1>(a, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv8_merge(const Kv8AttnArgs& a, cudaStream_t st) {
  const int64_t per = ((int64_t)a.prows * (a.hd / 4) + 31) / 32;
  const dim3 grid(cdiv((int64_t)a.B * a.units * per, 8)), block(256);
  switch (a.hd) {
    case 32: return launch_pdl(kv8_merge_kernel<32>, grid, block, 0, st, a);
    case 64: return launch_pdl(kv8_merge_kernel<64>, grid, block, 0, st, a);
    case 128: return launch_pdl(kv8_merge_kernel<128>, grid, block, 0, st, a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dg

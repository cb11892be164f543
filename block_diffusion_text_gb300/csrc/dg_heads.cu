// RMSNorm of the query and key heads with the position rotation, from the packed
// projection of a token, [q heads | k heads | v heads], into the layouts that
// attention and the cache's append take:
//
//   t = x g / sqrt(mean(x^2) + eps),  (a, b) -> (a cos - b sin, a sin + b cos)
//
// with a the first and b the second half of the head and the angle pos base^(-2 j / hd)
// for pair j; v heads are moved.  Bound by memory: every value is read once and
// written once (16384 tokens of 32 heads of 128: 48.8 us, 5.5 TB/s; one token 2 us).
#include <climits>
#include <cmath>

#include "dg_common.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kHeadThreads = 256;

// theta_j / (2 pi) as a 64-bit binary fraction of a turn.  The integer product
// with a position, modulo 2^64, is the angle in turns modulo one: no far position
// loses bits (an angle is off by pos 2^-54 theta / 2 pi at most, as a double's
// rounding of theta is).
struct HeadTurns {
  uint64_t t[64];
};

struct HeadArgs {
  const __nv_bfloat16* x;        // [B][C][W], strides sb, st
  const int* pos;                // [B]
  const __nv_bfloat16 *qg, *kg;  // [hd] or null
  __nv_bfloat16 *q, *k, *v;      // [B][H][C][hd]
  int64_t sb, st;
  int tokens;                    // B * C
  int C, Hq, Hkv;
  float eps;
};

// A thread holds eight pairs of one head: 16 bytes of its first half and 16 of
// its second.  A CTA takes `per` tokens, enough to fill its threads, and where there are
// many so many that each thread works out one sine and cosine, for all heads, while
// the first values are on their way; the next values are loaded before the last ones
// are worked on.  In shared memory the operands of neighbouring threads are neighbours,
// 16 bytes each: [quarter of the eight pairs][thread of the head].
template <int HD>
__global__ void __launch_bounds__(kHeadThreads) qk_norm_rope_kernel(HeadArgs a, HeadTurns turns, int per) {
  pdl_wait();
  constexpr int L = HD / 16;  // threads per head
  extern __shared__ __align__(16) float4 cs[];  // [per][4][L]: cosine and sine of two pairs
  __shared__ __align__(16) float4 gains[2][2][2][L];  // of q, k: [half of the head][half of the eight]
  const int H = a.Hq + 2 * a.Hkv, tid = threadIdx.x, items = H * L;
  const int tok0 = blockIdx.x * per, here = min(per, a.tokens - tok0);
  // where the thread stands: token of the CTA, its sequence and place, item of the token
  int ti = tid / items, item = tid - ti * items;
  int b = (tok0 + ti) / a.C, i = tok0 + ti - b * a.C;
  auto advance = [&]() {
    item += kHeadThreads;
    while (item >= items) {
      item -= items;
      ++ti;
      if (++i == a.C) {
        i = 0;
        ++b;
      }
    }
  };
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  auto load = [&]() {
    const uint4* src = reinterpret_cast<const uint4*>(a.x + b * a.sb + i * a.st + item / L * HD) + item % L;
    lo = __ldcs(src);
    hi = __ldcs(src + L);
  };
  if (ti < here) load();
  for (int e = tid; e < 2 * HD; e += kHeadThreads) {
    const __nv_bfloat16* from = e < HD ? a.qg : a.kg;
    const int j = e % (HD / 2);  // of the half: pair j is pair j % 8 of thread j / 8
    reinterpret_cast<float*>(&gains[e / HD][e / (HD / 2) % 2][j % 8 / 4][j / 8])[j % 4] = from ? __bfloat162float(from[e % HD]) : 1.0f;
  }
  for (int e = tid; e < here * (HD / 2); e += kHeadThreads) {
    const int tok = tok0 + e / (HD / 2), j = e % (HD / 2);
    const uint64_t at = (uint64_t)((int64_t)a.pos[tok / a.C] + tok % a.C);
    const int32_t turn = (int32_t)(uint32_t)((at * turns.t[j]) >> 32);  // signed: half a turn is 2^31
    float sn, c;
    sincospif((float)turn * 4.656612873077393e-10f, &sn, &c);  // 2^-31
    reinterpret_cast<float2*>(cs + (e / (HD / 2) * 4 + j % 8 / 2) * L + j / 8)[j % 2] = make_float2(c, sn);
  }
  __syncthreads();
  while (ti < here) {
    const int head = item / L, l = item % L, at = ti;
    const bool isq = head < a.Hq, isv = head >= a.Hq + a.Hkv;
    const int hh = isq ? head : head - a.Hq - (isv ? a.Hkv : 0);
    __nv_bfloat16* dst = isq ? a.q + (((int64_t)b * a.Hq + hh) * a.C + i) * HD : (isv ? a.v : a.k) + (((int64_t)b * a.Hkv + hh) * a.C + i) * HD;
    uint4* d4 = reinterpret_cast<uint4*>(dst) + l;
    const uint4 vl = lo, vh = hi;
    advance();
    if (ti < here) load();
    if (isv) {
      __stcs(d4, vl);
      __stcs(d4 + L, vh);
      continue;
    }
    const uint32_t wl[4] = {vl.x, vl.y, vl.z, vl.w}, wh[4] = {vh.x, vh.y, vh.z, vh.w};
    float x[8], y[8], sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = __uint_as_float(j % 2 ? wl[j / 2] & 0xffff0000u : wl[j / 2] << 16);
      y[j] = __uint_as_float(j % 2 ? wh[j / 2] & 0xffff0000u : wh[j / 2] << 16);
      sum += x[j] * x[j] + y[j] * y[j];
    }
    // a head's lanes are neighbours and come together: the items are a multiple of L
    const unsigned mask = ((1u << L) - 1) << (tid % 32 / L * L);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(mask, sum, o);
    const float inv = 1.0f / sqrtf(sum * (1.0f / HD) + a.eps);
    const float4(&gain)[2][2][L] = gains[isq ? 0 : 1];
    uint32_t ol[4], oh[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 g0 = gain[0][q][l], g1 = gain[1][q][l], c0 = cs[(at * 4 + 2 * q) * L + l], c1 = cs[(at * 4 + 2 * q + 1) * L + l];
      const float ga[4] = {g0.x, g0.y, g0.z, g0.w}, gb[4] = {g1.x, g1.y, g1.z, g1.w};
      const float cc[4] = {c0.x, c0.z, c1.x, c1.z}, sn[4] = {c0.y, c0.w, c1.y, c1.w};
      float u[4], w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = x[4 * q + e] * inv * ga[e], r = y[4 * q + e] * inv * gb[e];
        u[e] = p * cc[e] - r * sn[e];
        w[e] = p * sn[e] + r * cc[e];
      }
      ol[2 * q] = pack_bf16(u[0], u[1]);
      ol[2 * q + 1] = pack_bf16(u[2], u[3]);
      oh[2 * q] = pack_bf16(w[0], w[1]);
      oh[2 * q + 1] = pack_bf16(w[2], w[3]);
    }
    __stcs(d4, make_uint4(ol[0], ol[1], ol[2], ol[3]));
    __stcs(d4 + L, make_uint4(oh[0], oh[1], oh[2], oh[3]));
  }
}

// The table of a base and head dim; a host thread keeps the last one (64 powers take as
// long as the launch).
const HeadTurns& turns_of(float base, int hd) {
  thread_local HeadTurns t;
  thread_local float of_base = 0.f;
  thread_local int of_hd = 0;
  if (of_base != base || of_hd != hd) {
    t = HeadTurns{};
    for (int j = 0; j < hd / 2; ++j)
      t.t[j] = (uint64_t)std::ldexp(std::pow((double)base, -2.0 * j / hd) * 0.15915494309189535, 64);  // 1 / 2 pi
    of_base = base;
    of_hd = hd;
  }
  return t;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" dg_status dg_qk_norm_rope(const void* qkv, int64_t batch_stride, int64_t token_stride, const int32_t* pos,
                                     const void* q_gain, const void* k_gain, void* q, void* k, void* v, int32_t B,
                                     int32_t C, int32_t Hq, int32_t Hkv, int32_t hd, float rope_base, float rms_eps,
                                     void* stream) {
  if (!qkv || !pos || !q || !k || !v || B <= 0 || C <= 0 || Hq <= 0 || Hkv <= 0) return DG_ERR_ARG;
  if (!(rope_base >= 1.f) || !std::isfinite(rope_base) || !(rms_eps >= 0.f)) return DG_ERR_ARG;
  if (hd != 32 && hd != 64 && hd != 128) return DG_ERR_SHAPE;
  if (Hq > 1024 || Hkv > 1024 || (int64_t)B * C > (1 << 26)) return DG_ERR_SHAPE;
  const int64_t W = (int64_t)(Hq + 2 * Hkv) * hd;
  if ((C > 1 && token_stride < W) || token_stride % 8 || batch_stride % 8 || (B > 1 && batch_stride < W)) return DG_ERR_ARG;
  if (!aligned16(qkv) || !aligned16(q) || !aligned16(k) || !aligned16(v) || reinterpret_cast<uintptr_t>(pos) % 4 ||
      reinterpret_cast<uintptr_t>(q_gain) % 2 || reinterpret_cast<uintptr_t>(k_gain) % 2)
    return DG_ERR_ARG;
  const HeadTurns& turns = turns_of(rope_base, hd);
  HeadArgs a{static_cast<const __nv_bfloat16*>(qkv), pos, static_cast<const __nv_bfloat16*>(q_gain),
             static_cast<const __nv_bfloat16*>(k_gain), static_cast<__nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(k),
             static_cast<__nv_bfloat16*>(v), batch_stride, token_stride, B * C, C, Hq, Hkv, rms_eps};
  const int items = (Hq + 2 * Hkv) * (hd / 16);
  int per = items >= kHeadThreads ? 1 : kHeadThreads / items;
  // with many tokens, a sine and cosine for every thread (16 / 8 heads of 128: 608 tokens
  // 3.9 us against 3.2 without, 1216 4.9 against 5.2, 4096 12.4 against 16.5, 16384 48.8
  // against 64.9)
  const int fill = kHeadThreads / (hd / 2);
  if (per < fill && a.tokens >= 2 * kTargetCtas * fill) per = fill;
  const dim3 grid(cdiv(a.tokens, per)), block(kHeadThreads);
  const size_t smem = sizeof(float2) * per * (hd / 2);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = hd == 32   ? launch_pdl(qk_norm_rope_kernel<32>, grid, block, smem, st, a, turns, per)
                  : hd == 64 ? launch_pdl(qk_norm_rope_kernel<64>, grid, block, smem, st, a, turns, per)
                             : launch_pdl(qk_norm_rope_kernel<128>, grid, block, smem, st, a, turns, per);
  return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

// The 8-bit prefix cache: quantisation of rows as they are written, read-back,
// and the entry points of its attention.
//
// A cached row is hd E4M3 codes; a block of 64 rows of one (sequence, kv head)
// shares a power-of-two scale 2^e.  A power of two costs no relative precision
// (E4M3 is a floating-point format) and buys four things: the quotient x 2^-e
// is exact, so a code is the correctly rounded value; code x scale is exact in
// bf16; a block whose scale grows moves its codes without a second rounding
// (but for subnormals); and attention can fold scales into exponents.
#include <climits>

#include "dg_kv8.cuh"

namespace dg {
namespace {

// ----------------------------------------------------------------- append --
struct Kv8AppendArgs {
  const void *k, *v;      // bf16 [B][Hkv][n][hd]
  uint8_t *K, *V, *Ke, *Ve;
  const int *len, *counts;
  int* status;
  int B, n, Hkv, hd, cap, nblk;
};

constexpr int kAppendThreads = 256;

// One CTA per (block of 64 cached rows, kv head and sequence, K or V): the new
// rows that fall into the block stay in registers between the reduction of
// their maximum and the rounding, so every input is read once.  16 values per
// thread and chunk: two 16-byte loads, one 16-byte store.  Bound by memory: 4
// sequences of 16384 rows and 8 heads 59.0 us (floor at the measured copy rate
// 59.2); one row each of 32 sequences 2.5 us, a launch.
template <int HD>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(Kv8AppendArgs a) {
  pdl_wait();
  constexpr int CPR = HD / 16;                                   // chunks per row
  constexpr int NCH = kKv8Block * CPR;
  constexpr int PER = (NCH + kAppendThreads - 1) / kAppendThreads;
  __shared__ unsigned red[kAppendThreads / 32];
  const int bh = blockIdx.y, b = bh / a.Hkv, tid = threadIdx.x;
  const bool isv = blockIdx.z != 0;
  const int len = a.len[b], n = a.counts ? a.counts[b] : a.n;
  if (len < 0 || n < 0 || n > a.n || (long long)len + n > a.cap) {  // nothing of this sequence is written
    if (tid == 0) atomicExch(a.status, (n < 0 || n > a.n) ? kStatusArg : kStatusCapacity);
    return;
  }
  const int blk = len / kKv8Block + blockIdx.x;
  const int row0 = blk * kKv8Block;                              // first cached row of the block
  const int lo = max(len - row0, 0), hi = min(len + n - row0, kKv8Block);  // its new rows
  if (hi <= lo) return;
  const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(isv ? a.v : a.k) + (size_t)bh * a.n * HD;
  uint8_t* dst = (isv ? a.V : a.K) + ((size_t)bh * a.cap + row0) * HD;
  uint8_t* ep = (isv ? a.Ve : a.Ke) + (size_t)bh * a.nblk + blk;

  uint4 x[PER][2];
  unsigned top = 0;                                              // two 16-bit maxima of |x|'s bits
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int c = p * kAppendThreads + tid, r = c / CPR;
    const bool mine = c < NCH && r >= lo && r < hi;
    x[p][0] = x[p][1] = make_uint4(0, 0, 0, 0);
    if (mine) {
      const uint4* s = reinterpret_cast<const uint4*>(src + (size_t)(row0 + r - len) * HD + (c % CPR) * 16);
      x[p][0] = __ldcs(s);
      x[p][1] = __ldcs(s + 1);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) top = __vmaxu2(top, abs_top(x[p][h]));
  }
  auto block_max = [&](unsigned t) {
    t = max(t & 0xffffu, t >> 16);
    t = __reduce_max_sync(0xffffffffu, t);
    if (tid % 32 == 0) red[tid / 32] = t;
    __syncthreads();
    t = red[tid % (kAppendThreads / 32)];
    return __reduce_max_sync(0xffffffffu, t);
  };
  unsigned amax = block_max(top);
  if (amax >= 0x7f80u) {
    // An infinity or NaN among the values: the scale goes by the finite ones,
    // infinities saturate, NaN is stored as zero, and the status word says so.
    if (tid == 0) atomicExch(a.status, kStatusValue);
    top = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&x[p][0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const unsigned mag = (w[j] >> (16 * h)) & 0x7fffu;
          if (mag > 0x7f80u) w[j] &= ~(0xffffu << (16 * h));
          if (mag < 0x7f80u) top = max(top, mag);
        }
      }
    }
    __syncthreads();  // red is read above
    amax = block_max(top);
  }
  int e = top_exponent(amax);
  if (lo > 0) {
    // Earlier rows share the block: its scale never shrinks, and where it
    // grows their codes move to it.
    const int was = (int)*ep - kKv8Bias;
    if (e > was) {
      const float f = pow2i(was - e);
      for (int c = tid; c < lo * CPR; c += kAppendThreads) {
        uint4 w = *reinterpret_cast<const uint4*>(dst + c * 16);
        uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t h0 = e4m3x2_f16x2(u[j]), h1 = e4m3x2_f16x2(u[j] >> 16);
          const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
          const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
          u[j] = pack_e4m3(f0.x * f, f0.y * f) | (pack_e4m3(f1.x * f, f1.y * f) << 16);
        }
        *reinterpret_cast<uint4*>(dst + c * 16) = w;
      }
    } else {
      e = was;
    }
    __syncthreads();  // every thread has read *ep
  }
  if (tid == 0) *ep = (uint8_t)(e + kKv8Bias);
  const float f = pow2i(-e);
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int c = p * kAppendThreads + tid, r = c / CPR;
    if (c >= NCH || r < lo || r >= hi) continue;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[p][0]);
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = w[2 * j], t = w[2 * j + 1];
      q[j] = pack_e4m3(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xffff0000u) * f) |
             (pack_e4m3(__uint_as_float(t << 16) * f, __uint_as_float(t & 0xffff0000u) * f) << 16);
    }
    *reinterpret_cast<uint4*>(dst + c * 16) = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

// ------------------------------------------------------------------- read --
struct Kv8ReadArgs {
  const uint8_t *K, *V, *Ke, *Ve;
  const int* len;
  void *k, *v;            // bf16 [B][Hkv][pitch][hd]
  int* status;
  int B, Hkv, hd, cap, nblk, row0, n, pitch;
  int wide;               // k and v aligned to 32 bytes
};

constexpr int kReadThreads = 128;

// Codes back to bf16 (exact): 16 codes per thread, one 16-byte load and one
// 32-byte store (a whole sector; two of 16 bytes where an output is not aligned
// to 32).  Bound by memory, two thirds of it the writes: 131072 rows of 8 heads
// 118.0 us (the floor at the measured copy rate is 118.5), with the two stores
// 121.2, with four chunks a thread and 256 threads 127.1.
template <int HD>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(Kv8ReadArgs a) {
  pdl_wait();
  constexpr int CPR = HD / 16;
  const int bh = blockIdx.y, b = bh / a.Hkv;
  const bool isv = blockIdx.z != 0;
  const int len = a.len[b];
  if ((len < 0 || len > a.cap) && blockIdx.x == 0 && threadIdx.x == 0) atomicExch(a.status, kStatusCapacity);
  const int rows = min(a.n, min(max(len, 0), a.cap) - a.row0);   // rows of this sequence in the range (no length overflows)
  const long long c = (long long)blockIdx.x * kReadThreads + threadIdx.x;
  const int row = (int)(c / CPR);
  if (row >= rows) return;
  const uint8_t* src = (isv ? a.V : a.K) + ((size_t)bh * a.cap + a.row0) * HD;
  const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src + c * 16));
  const float f = pow2i((int)((isv ? a.Ve : a.Ke) + (size_t)bh * a.nblk)[(a.row0 + row) / kKv8Block] - kKv8Bias);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t h = e4m3x2_f16x2(u[j / 2] >> (16 * (j & 1)));
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[j] = pack_bf16(t.x * f, t.y * f);
  }
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(isv ? a.v : a.k) + (size_t)bh * a.pitch * HD + c * 16;
  if (a.wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                 "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                 : "memory");
  } else {
    uint4* d = reinterpret_cast<uint4*>(dst);
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The checks every entry point of the cache shares.
dg_status check_kv8(const dg_kv8_cache* c) {
  if (!c || !c->K || !c->V || !c->K_exp || !c->V_exp || !c->len || !c->status) return DG_ERR_ARG;
  if (c->B <= 0 || c->Hkv <= 0 || c->cap <= 0) return DG_ERR_ARG;
  if (!aligned16(c->K) || !aligned16(c->V)) return DG_ERR_ARG;
  if (c->hd != 32 && c->hd != 64 && c->hd != 128) return DG_ERR_SHAPE;
  // grid.y holds one row per (sequence, kv head); TMA row coordinates are int32
  if ((int64_t)c->B * c->Hkv > 65535 || (int64_t)c->B * c->Hkv * c->cap > INT32_MAX - 65536 || c->cap > (1 << 30))
    return DG_ERR_SHAPE;
  return DG_OK;
}

dg_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DG_OK : DG_ERR_CUDA; }

int kv8_blocks(int cap) { return cdiv(cap, kKv8Block); }

// Key tiles to a CTA (and to a warp of its groups), above which shares balance better than they
// cost: 8 ragged sequences of up to 8000 rows, 8 heads, 15.2 us in shares, 19.5 with
// two CTAs a unit; up to 4000 rows 13.2 against 12.6.
constexpr int kClusterTiles = 64, kGroupTiles = 16;
constexpr int kKv8Ovh = 3;  // measured: a unit's start and output take as long as some three tiles

// CTAs that share a unit of `tiles` key tiles, of `units` in the call: as many
// as give every warp half a tile, while all clusters run at once (what
// cudaOccupancyMaxActiveClusters answers for clusters of 2 to 8 CTAs of the
// warp-MMA kernel, one to an SM; a second wave costs more: 16 units of 4000 rows
// 14.2 us with 8 CTAs each, 8.3 with 6), one where its own warps suffice.
int kv8_cluster(int64_t units, int tiles, int warps) {
  constexpr int kFit[kMaxCluster + 1] = {0, 0, 76, 46, 36, 28, 23, 15, 15};
  int n = 1;
  if (tiles > warps)
    while (n < kMaxCluster && n * warps < 2 * tiles && units <= kFit[n + 1]) ++n;
  return n;
}

struct Kv8Ws {
  size_t part, ml, total;
  int rows, tk, units, workers, prows, subs, cluster, group;
  bool tc;
};

// The kernel, its rows per unit, and the workspace of an attention call.
Kv8Ws kv8_ws(const dg_kv8_cache* c, int C, int Hq) {
  Kv8Ws w{};
  const int64_t R = (int64_t)(Hq / c->Hkv) * C;
  const int tiles = cdiv(c->cap, kKv8Block) + cdiv(C, kKv8Block);
  // The tensor-core kernel takes more than 16 rows, but for calls that the warps
  // finish in one launch and one wave with a few tiles each (new tokens' tiles
  // take a warp twice as long): 64 query rows to a head, 4000 rows, 8 heads 14.1 us
  // against 14.4; 256 rows, 1500 rows, 2 heads 12.3 against 14.6; with more tiles
  // to a warp it turns: 64 rows, 8000 rows, 16 heads 27.1 against 25.3, 256 rows,
  // 2000 rows, 4 heads 19.9 against 16.0 (head dim 128; with 64, 128 rows, 6000 rows,
  // 4 heads 15.7 and 13.3).  Head dim 32, half a row of a swizzled tile and no
  // workload's but the smallest, stays with the warps.  All of this goes by the
  // capacity: the lengths are the device's.
  const int rows = kv8_mma_rows(c->hd, R), warps = kv8_mma_warps(c->hd, rows);
  const int64_t all = (int64_t)c->B * c->Hkv * ((R + rows - 1) / rows);
  const int cluster = kv8_cluster(all, tiles, warps);
  // With more units than SMs the tensor-core kernel, which begins and ends a CTA's
  // units one after another, loses on short ones: 400 heads of 24 rows over up to 500
  // rows 41.1 us against 34.6, over up to 1000 49.5 against 87.0; of 64 rows, 8 tokens of
  // 8 heads, over up to 250 rows 44.7 against 40.7, over up to 500 47.7 against 52.2.
  // (Of 64 tokens it turns earlier, 250 rows 45.5 against 51.9: still the warps'.)
  const bool few = all <= kKv8Ctas ? tiles <= (C <= kKv8Block ? 4 : 1) * cluster * warps
                                   : C <= kKv8Block && tiles * ((R + rows - 1) / rows) < 32;
  w.tc = c->hd >= 64 && R > 16 && !few;
  w.subs = w.tc && R <= 128 ? 2 : 1;  // one row tile is enough: the two take every other key tile
  w.rows = w.tc ? 256 / w.subs : rows;
  w.tk = w.tc ? 128 : kKv8Block;
  w.workers = w.tc ? kKv8Ctas : kKv8Ctas * warps;
  w.units = (int)(c->Hkv * ((R + w.rows - 1) / w.rows));  // at most 65535 * 64 by the checks before
  w.prows = (int)(R < w.rows ? R : w.rows);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  if (!w.tc) {
    // A short cache's units are finished by a cluster of CTAs each, without parts
    // in memory and a merge kernel.  One token of one sequence, 2 kv heads, with
    // and without: 4000 rows 7.5 and 9.4 us, 8000 9.6 and 12.1, 32000 20.0 and
    // 28.4; 8 heads 32000 rows 20.0 and 21.1.
    // More units than SMs share CTAs, each a group of the warps: 64 sequences of
    // up to 500 rows, 8 heads, 10 us, one CTA to each 19; 500 sequences of up to 250
    // rows 55 us, 152 with a CTA to each, 140 in shares.
    int group = warps;
    if (cluster == 1)
      while (group > 1 && cdiv(all, warps / group) > kKv8Ctas)
        do --group;
        while (warps % group);
    if (tiles <= (group == warps ? kClusterTiles * cluster : 2 * group == warps ? 40 : kGroupTiles * group)) {
      w.cluster = cluster;
      w.group = group;
      return w;
    }
  }
  w.part = take((size_t)2 * w.workers * w.subs * w.prows * c->hd * 4);
  w.ml = take((size_t)2 * w.workers * w.subs * w.prows * 8);
  w.total = off;
  return w;
}

dg_status check_kv8_attention(const dg_kv8_cache* c, int C, int Hq) {
  dg_status s = check_kv8(c);
  if (s) return s;
  if (C <= 0 || Hq <= 0 || Hq % c->Hkv != 0) return DG_ERR_ARG;
  // the bounds the denoising step and dg_attention_noalloc apply
  if (C > 1024 || (int64_t)c->B * C > (1 << 20) || (int64_t)c->B * Hq > 65535) return DG_ERR_SHAPE;
  // tiles, and CTAs of the merge, are counted in 32 bits
  const Kv8Ws w = kv8_ws(c, C, Hq);
  const int64_t tiles = (int64_t)c->B * w.units * (cdiv(c->cap, w.tk) + cdiv(C, w.tk) + kKv8Ovh);
  const int64_t ctas = (int64_t)c->B * w.units * cdiv((int64_t)w.prows * c->hd, 128);
  if (tiles > INT32_MAX - 65536 || ctas > INT32_MAX - 65536) return DG_ERR_SHAPE;
  return DG_OK;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" dg_status dg_kv8_append(const dg_kv8_cache* cache, const void* k, const void* v, int32_t n,
                                   const int32_t* counts, void* stream) {
  dg_status s = check_kv8(cache);
  if (s) return s;
  if (!k || !v || n <= 0 || !aligned16(k) || !aligned16(v)) return DG_ERR_ARG;
  if (n > cache->cap) return DG_ERR_CAPACITY;
  Kv8AppendArgs a{k, v, static_cast<uint8_t*>(cache->K), static_cast<uint8_t*>(cache->V),
                  static_cast<uint8_t*>(cache->K_exp), static_cast<uint8_t*>(cache->V_exp), cache->len, counts,
                  cache->status, cache->B, n, cache->Hkv, cache->hd, cache->cap, kv8_blocks(cache->cap)};
  // blocks that n rows can touch, from any offset
  const dim3 grid((n - 1 + kKv8Block - 1) / kKv8Block + 1, cache->B * cache->Hkv, 2);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (cache->hd) {
    case 32: return from_cuda(launch_pdl(kv8_append_kernel<32>, grid, dim3(kAppendThreads), 0, st, a));
    case 64: return from_cuda(launch_pdl(kv8_append_kernel<64>, grid, dim3(kAppendThreads), 0, st, a));
  }
  return from_cuda(launch_pdl(kv8_append_kernel<128>, grid, dim3(kAppendThreads), 0, st, a));
}

extern "C" dg_status dg_kv8_read(const dg_kv8_cache* cache, int32_t row0, int32_t n, void* k, void* v,
                                 int32_t pitch, void* stream) {
  dg_status s = check_kv8(cache);
  if (s) return s;
  if (!k || !v || row0 < 0 || n <= 0 || pitch < n || !aligned16(k) || !aligned16(v)) return DG_ERR_ARG;
  if (row0 >= cache->cap) return DG_OK;  // no row there: nothing to write
  Kv8ReadArgs a{static_cast<const uint8_t*>(cache->K), static_cast<const uint8_t*>(cache->V),
                static_cast<const uint8_t*>(cache->K_exp), static_cast<const uint8_t*>(cache->V_exp), cache->len, k, v,
                cache->status, cache->B, cache->Hkv, cache->hd, cache->cap, kv8_blocks(cache->cap), row0, n, pitch,
                (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 32 == 0};
  const int rows = n < cache->cap - row0 ? n : cache->cap - row0;
  const dim3 grid(cdiv((int64_t)rows * (cache->hd / 16), kReadThreads), cache->B * cache->Hkv, 2);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (cache->hd) {
    case 32: return from_cuda(launch_pdl(kv8_read_kernel<32>, grid, dim3(kReadThreads), 0, st, a));
    case 64: return from_cuda(launch_pdl(kv8_read_kernel<64>, grid, dim3(kReadThreads), 0, st, a));
  }
  return from_cuda(launch_pdl(kv8_read_kernel<128>, grid, dim3(kReadThreads), 0, st, a));
}

extern "C" dg_status dg_kv8_attention_workspace(const dg_kv8_cache* cache, int32_t C, int32_t Hq, size_t* bytes) {
  if (!bytes) return DG_ERR_ARG;
  dg_status s = check_kv8_attention(cache, C, Hq);
  if (s) return s;
  *bytes = kv8_ws(cache, C, Hq).total;
  return DG_OK;
}

extern "C" dg_status dg_kv8_attention(const dg_kv8_cache* cache, const void* q, const void* k, const void* v, void* o,
                                      int32_t C, int32_t Hq, int32_t causal, void* ws, size_t ws_bytes,
                                      void* stream) {
  dg_status s = check_kv8_attention(cache, C, Hq);
  if (s) return s;
  if (!q || !o || !k != !v) return DG_ERR_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(k) || !aligned16(v)) return DG_ERR_ARG;
  const Kv8Ws w = kv8_ws(cache, C, Hq);
  if (w.total > 0 && !ws) return DG_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < w.total) return DG_ERR_WORKSPACE;
  uint8_t* base = static_cast<uint8_t*>(ws);
  Kv8AttnArgs a{};
  a.q = q;
  a.K = static_cast<const uint8_t*>(cache->K);
  a.V = static_cast<const uint8_t*>(cache->V);
  a.Ke = static_cast<const uint8_t*>(cache->K_exp);
  a.Ve = static_cast<const uint8_t*>(cache->V_exp);
  a.len = cache->len;
  a.kn = k;
  a.vn = v;
  a.o = o;
  a.part = reinterpret_cast<float*>(base + w.part);
  a.ml = reinterpret_cast<float2*>(base + w.ml);
  a.status = cache->status;
  a.B = cache->B;
  a.C = C;
  a.Hq = Hq;
  a.Hkv = cache->Hkv;
  a.hd = cache->hd;
  a.cap = cache->cap;
  a.nblk = kv8_blocks(cache->cap);
  a.causal = causal != 0;
  a.rows = w.rows;
  a.tk = w.tk;
  a.units = w.units;
  a.workers = w.workers;
  a.ovh = kKv8Ovh;
  a.subs = w.subs;
  a.prows = w.prows;
  a.cluster = w.cluster;
  a.group = w.group;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = w.tc ? launch_kv8_attention_tc(a, st) : launch_kv8_attention_mma(a, st);
  if (e == cudaSuccess && !w.cluster) e = launch_kv8_merge(a, st);
  return from_cuda(e);
}

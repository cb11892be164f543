// Tensor-core (tcgen05 + TMA) attention over the 8-bit prefix cache for many
// query rows per kv head (canvases and prompt pieces), head dims 64 and 128.
//
// A CTA owns 256 query rows (two tiles of 128) of one (sequence, kv head) and a
// run of 128-key tiles; the tiles of a call are dealt to the CTAs in equal
// shares (dg_kv8.cuh), parts are merged by kv8_merge_kernel.  What the 8-bit
// cache changes against the bf16 kernel (dg_attn_tc.cu):
//  - S = Q K^T runs on kind::f8f6f4, so the key codes go from TMA into the MMA
//    as they lie in memory.  A query row is split into two E4M3 terms, q 2^-x =
//    hi + lo: a bf16 has 8 significant bits and each term holds 4, so the split
//    is exact for elements down to 2^-10 of the row's largest and off by
//    2^-10 / 224 of the largest below (its own bf16 rounding is 2^-9 of each).
//    Two products at twice the 16-bit rate cost what one 16-bit product costs.
//  - P V runs in f16: p' is rounded to f16 (2^-12), once, where bf16 would need
//    two terms; the value codes become f16 (exact) in shared memory, by four
//    warps that do nothing else.
//  - Block scales never touch the codes: 2^ke joins the softmax factor of its 64
//    columns and 2^ve the exponent of the probability (the running maximum is
//    that of s + ve), whose share of the row sum is taken back.
// The new tokens' bf16 keys and values are brought into the same forms by
// kv8_prep_kernel: keys as two E4M3 terms on a scale per 64 tokens (four
// products), values as f16 on such a scale (exact to 2^-22 of the block's
// largest).
//
// Warp roles (16 warps, one CTA per SM):
//   warp 0       TMA: Q terms per piece, K tiles into a ring of slots (a new tile
//                takes two), V codes into their own ring (new tiles:
//                f16, straight to the MMA's buffer)
//   warps 1, 2   MMA, one for each row tile, taking turns: P_t V of key tile j, then
//                S_t of tile j + 1, so that one row tile's softmax and waits run
//                under the other's products
//   warps 4-7    V codes to f16
//   warps 8-15   softmax, one thread per row; P over S in TMEM
//
// Measured: a canvas of 256 rows over 131072 rows of 8 heads 116 us (the two
// products at the measured bf16 rate: 72), 1.18 PFLOP/s; a key tile takes 3640
// cycles, 2048 of them MMAs.  A row tile's chain (scores ready, two passes of
// softmax 2100 to 2300 cycles, P V and the next S 1250) bounds it: without the
// exponentials it runs 107 us, without all softmax work 83.  Tried and slower:
// two threads a row (24 warps of 80 registers, 123 us; 20 of 96, 168 us), the
// scores read once block by block (123 to 129), the probabilities made on the old
// maximum in one pass and again where it grew (135), loads 32 columns ahead (129),
// scores of 64 keys at a time, two of them in flight to a row tile (126 to 129:
// the softmax no longer waits, but an MMA of 64 columns takes as long as one of
// 128 and the MMA warps have twice the turns), MMA warps without turns (143).
// Head dim 64 has half the MMAs and the same softmax: 256 rows over 32768 rows of
// 8 heads 35.3 us (head dim 128: 42.6; the warp-MMA kernel 91.7).
#include <cfloat>

#include "dg_kv8.cuh"

namespace dg {
namespace {

constexpr int kTK = 128;                   // keys per tile
constexpr int kThreads = 512;
constexpr int kNK = 4, kNV = 2;            // ring depths: K slots, V code and f16 slots
constexpr float kHeadroom = 8.0f;          // p' of a row's maximum is 2^8 ..
constexpr float kLazy = 6.0f;              // .. to 2^14: O is rescaled when the maximum grew by more than 2^6

template <int HD>
struct Smem {
  static constexpr int kQ = 128 * HD;                // one term of one row tile
  static constexpr int kK = kTK * HD;                // one tile of codes
  static constexpr int kBox = kTK * 128;             // 64 f16 columns of a tile
  static constexpr int kF16 = HD / 64 * kBox;
  static constexpr int oK = 4 * kQ;
  static constexpr int oVc = oK + kNK * kK;
  static constexpr int oVf = oVc + kNV * kK;
  static constexpr int oBar = oVf + kNV * kF16;
  static constexpr int oMl = oBar + 512;             // float2 [2 row tiles][128]: maximum and sum
  static constexpr int oFrom = oMl + 2 * 128 * 8;    // int2 [warps]: kv8_piece's `from`
  static constexpr int kTotal = oFrom + kThreads / 32 * 8;
  static_assert(kTotal <= 232448, "shared memory of one CTA");
};

// TMEM: S_t at 128 t (P_t over its first 64 columns), O_t at 256 + 128 t.
constexpr int kColO = 256;

// An MMA warp runs as one: every lane reaches these, one elected lane issues.
// With the election inside, the descriptors stay in uniform registers: 39
// cycles an MMA from issue to issue against 57 in a branch of lane 0 alone
// (measured alone; an MMA of this kernel takes the tensor core 64).
DG_DEV void mma_s(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum)
      : "memory");
}
DG_DEV void mma_pv(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accum)
      : "memory");
}
DG_DEV void commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}
// Shared-memory descriptors (swizzle over rows of SW bytes, 128 or 64, 8 SW bytes
// between 8-row groups) as a low word, address and leading offset, and a high word.
DG_DEV uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3FFFFu) >> 4) | (lbo >> 4 << 16); }
template <int SW>
DG_DEV uint64_t desc64(uint32_t lo) {
  constexpr uint32_t hi = (8u * SW >> 4) | (1u << 14) | ((SW == 128 ? 2u : 4u) << 29);
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "n"(hi));
  return d;
}
// D (+)= (Q_hi + Q_lo) K^T: the two terms of a query tile lie behind one another.
template <int HD>
DG_DEV void s_terms(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc, uint32_t accum) {
#pragma unroll
  for (int term = 0; term < 2; ++term)
#pragma unroll
    for (int kk = 0; kk < HD / 32; ++kk)
      mma_s(d, desc64<HD>(q + term * (Smem<HD>::kQ >> 4) + 2 * kk), desc64<HD>(k + 2 * kk), idesc, (term | kk) ? 1u : accum);
}
// Bounded wait of a whole warp whose usual case, the phase is complete, costs
// one try (63 cycles against 171 for mbar_wait_warp's loops, measured alone).
DG_DEV bool wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return mbar_wait_warp(bar, parity, status, abort);
}
DG_DEV void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One piece of a CTA's share: tiles t0..t1-1 of one unit.
struct Piece {
  int b, hk, row0, len, t0, t1, nt, ntc;
  DG_DEV int tiles() const { return t1 - t0; }
  DG_DEV bool fresh(int j) const { return t0 + j >= ntc; }  // tile j of the piece holds new tokens
};
// The next piece with tiles at or after w, or false.
DG_DEV bool next_piece(const Kv8AttnArgs& a, const Kv8Plan& plan, int2& from, int& w, int w1, Piece& p) {
  while (w < w1) {
    const Kv8Piece k = kv8_piece(a, plan, from, w, w1);
    w += k.cost;
    if (k.t1 <= k.t0) continue;
    const int per = a.units / a.Hkv;
    p = Piece{k.b, k.unit / per, k.unit % per * a.rows, k.len, k.t0, k.t1, k.nt, (k.len + kTK - 1) / kTK};
    return true;
  }
  return false;
}

// DUP: up to 128 query rows.  Both row tiles hold the same rows and row tile t
// takes key tiles t, t + 2, ..; their outputs are two parts, which the softmax
// warps join themselves where the CTA has all of the unit's tiles.
template <int HD, bool DUP>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_attn_tc_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                       const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mKn,
                       const __grid_constant__ CUtensorMap mVn, Kv8AttnArgs a, Kv8Prep pp, float scale_log2) {
  using Smem = Smem<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {  // uniform over the CTA: return before any barrier
    if (threadIdx.x == 0) atomicExch(a.status, kStatusTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::oBar);
  uint64_t* qfull = bars;
  uint64_t* qempty = qfull + 1;
  uint64_t* kfull = qempty + 1;      // [kNK]
  uint64_t* kempty = kfull + kNK;    // [kNK]
  uint64_t* cfull = kempty + kNK;    // [kNV] V codes (or new f16 values) have landed
  uint64_t* cempty = cfull + kNV;    // [kNV] V codes have been read
  uint64_t* vfull = cempty + kNV;    // [kNV] f16 values ready for the MMA
  uint64_t* vempty = vfull + kNV;    // [kNV]
  uint64_t* sfull = vempty + kNV;    // [2]
  uint64_t* pready = sfull + 2;      // [2 tiles][2 halves]
  uint64_t* pvdone = pready + 4;     // [2]
  uint64_t* turn = pvdone + 2;       // [2] row tile t's MMA warp may issue
  uint64_t* meet = turn + 2;         // the softmax warps of both row tiles
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meet + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* status = a.status;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(qfull, 1);
    constexpr int readers = DUP ? 1 : 2;  // MMA warps that read a tile
    mbar_init(qempty, 2);
    mbar_init(meet, 8);
    for (int s = 0; s < kNK; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], readers);
    }
    for (int s = 0; s < kNV; ++s) {
      mbar_init(&cfull[s], 1);
      mbar_init(&cempty[s], 4);
      mbar_init(&vfull[s], 4);
      mbar_init(&vempty[s], readers);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pready[2 * t], 4);
      mbar_init(&pready[2 * t + 1], 4);
      mbar_init(&pvdone[t], 1);
      mbar_init(&turn[t], 1);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();  // the merge, which needs no TMEM, may take the SMs that this kernel leaves

  const Kv8Plan plan = kv8_plan(a);
  int2& from = reinterpret_cast<int2*>(smem + Smem::oFrom)[warp];  // in memory: registers are short
  from = make_int2(0, 0);
  __syncwarp();
  const int w0 = (int)min((long long)plan.total, (long long)blockIdx.x * plan.share);
  const int w1 = (int)min((long long)plan.total, (long long)w0 + plan.share);
  const int grp_rows = a.Hq / a.Hkv * a.C;

  if (warp < 4) {
    if (warp == 0) {
      if (blockIdx.x == 0)
        for (int b = lane; b < a.B; b += 32)
          if (a.len[b] < 0 || a.len[b] > a.cap) atomicExch(status, kStatusCapacity);
      if (lane == 0) {
        tma_prefetch(&mQ);
        tma_prefetch(&mK);
        tma_prefetch(&mV);
      }
      bool ok = true;
      int kslot = 0, kpar = 1, J = 0, np = 0;  // slot counters run on through the pieces
      Piece p;
      for (int w = w0; ok && next_piece(a, plan, from, w, w1, p); ++np) {
        if (lane == 0) {
          const int bh = p.b * a.Hkv + p.hk;
          ok = mbar_wait(qempty, (np & 1) ^ 1, status, abort);
          if (ok) {
            const int qrow = bh * grp_rows + p.row0;
            mbar_arrive_expect_tx(qfull, 4 * Smem::kQ);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int term = 0; term < 2; ++term)
                tma_load_2d(smem + (2 * t + term) * Smem::kQ, &mQ, qfull, 0, term * pp.qrows + qrow + (DUP ? 0 : 128 * t));
          }
          for (int j = 0; j < p.tiles() && ok; ++j, ++J) {
            const bool fresh = p.fresh(j);
            const int key = (p.t0 + j - (fresh ? p.ntc : 0)) * kTK;
            for (int term = 0; term < (fresh ? 2 : 1) && ok; ++term) {
              if (!(ok = mbar_wait(&kempty[kslot], kpar, status, abort))) break;
              mbar_arrive_expect_tx(&kfull[kslot], Smem::kK);
              tma_load_2d(smem + Smem::oK + kslot * Smem::kK, fresh ? &mKn : &mK, &kfull[kslot], 0,
                          fresh ? term * pp.krows + bh * pp.Cp + key : bh * a.cap + key);
              if (++kslot == kNK) {
                kslot = 0;
                kpar ^= 1;
              }
            }
            if (!ok) break;
            const int s = J % kNV, par = ((J / kNV) & 1) ^ 1;
            if (!(ok = mbar_wait(&cempty[s], par, status, abort))) break;
            if (fresh) {
              if (!(ok = mbar_wait(&vempty[s], par, status, abort))) break;
              uint8_t* dst = smem + Smem::oVf + s * Smem::kF16;
              mbar_arrive_expect_tx(&cfull[s], Smem::kF16);
              tma_load_2d(dst, &mVn, &cfull[s], 0, bh * pp.Cp + key);
              if (HD == 128) tma_load_2d(dst + Smem::kBox, &mVn, &cfull[s], 64, bh * pp.Cp + key);
            } else {
              mbar_arrive_expect_tx(&cfull[s], Smem::kK);
              tma_load_2d(smem + Smem::oVc + s * Smem::kK, &mV, &cfull[s], 0, bh * a.cap + key);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
    } else if (warp < 3) {
      const int t = warp - 1;
      constexpr uint32_t idS = idesc_e4m3(128, kTK);
      constexpr uint32_t idPV = idesc_f16(128, HD, true);
      const uint32_t lo_q = desc_lo(smem_u32(smem + 2 * t * Smem::kQ), 16), lo_k = desc_lo(smem_u32(smem + Smem::oK), 16);
      const uint32_t lo_v = desc_lo(smem_u32(smem + Smem::oVf), Smem::kBox);
      const uint32_t tS = tmem + 128 * t, tO = tmem + kColO + 128 * t;
      bool ok = true;
      static_assert((kNK & (kNK - 1)) == 0 && kNV == 2, "slots from running counts");
      int K = 0, J = 0, Jt = 0, np = 0, turns = t ^ 1;  // K slots, tiles, own tiles, pieces so far; parity of the turn
      const int stride = DUP ? 2 : 1, begin = DUP ? t : 0;
      Piece p;
      for (int w = w0; ok && next_piece(a, plan, from, w, w1, p); ++np) {
        const int n = p.tiles(), jfresh = max(p.ntc - p.t0, 0);  // tiles from jfresh on hold new tokens
        const int own = DUP ? (n + 1 - t) >> 1 : n, steps = DUP ? (n + 1) >> 1 : n;
        int j = begin - stride;                           // own key tile k of the piece
        int kc = K + (begin > 0 ? (jfresh > 0 ? 1 : 2) : 0);  // K slot of tile j + stride
        ok = wait(qfull, np & 1, status, abort);
        // Step k: P_t V of own key tile k, then S_t of own tile k + 1.  The two warps
        // take turns, step by step, which keeps the row tiles' softmax phases apart
        // (left alone they fall into step, and the tensor core idles while both
        // wait); each does its waiting and committing during the other's turn.
        // A commit covers all MMAs of its thread before it, so S_t of tile k + 1
        // also says that P_t V of tile k is done.
#pragma unroll 1
        for (int k = -1; k < steps && ok; ++k) {
          const int s = (J + j) & 1, jn = j + stride;
          const bool next = k + 1 < own, fresh = jn >= jfresh;
          const int ka = kc & (kNK - 1), kb = (kc + 1) & (kNK - 1);
          if (next) {
            if (!(ok = wait(&kfull[ka], (kc / kNK) & 1, status, abort))) break;
            if (fresh && !(ok = wait(&kfull[kb], ((kc + 1) / kNK) & 1, status, abort))) break;
          }
          if (k >= 0 && k < own) {
            if (!(ok = wait(&vfull[s], ((J + j) >> 1) & 1, status, abort))) break;
            // (the first P of a piece also says that the last one's output has been read)
            if (!(ok = wait(&pready[2 * t], (Jt + k) & 1, status, abort))) break;
            if (!(ok = wait(&turn[t], turns, status, abort))) break;
            tc_fence_after();
            const uint32_t v = lo_v + s * (Smem::kF16 >> 4);
#pragma unroll
            for (int k4 = 0; k4 < kTK / 32; ++k4)
              mma_pv(tO, tS + 8 * k4, desc64<128>(v + k4 * (2048 >> 4)), idPV, (k | k4) ? 1u : 0u);
            if (!(ok = wait(&pready[2 * t + 1], (Jt + k) & 1, status, abort))) break;
            tc_fence_after();
#pragma unroll
            for (int k4 = kTK / 32; k4 < kTK / 16; ++k4)
              mma_pv(tO, tS + 8 * k4, desc64<128>(v + k4 * (2048 >> 4)), idPV, 1u);
          } else {
            if (!(ok = wait(&turn[t], turns, status, abort))) break;
            tc_fence_after();
          }
          turns ^= 1;
          if (next) {
            uint32_t kd = lo_k + ka * (Smem::kK >> 4);
#pragma unroll 1
            for (int term = 0; term <= (fresh ? 1 : 0); ++term, kd = lo_k + kb * (Smem::kK >> 4))
              s_terms<HD>(tS, lo_q, kd, idS, term);
          }
          if (lane == 0) mbar_arrive(&turn[t ^ 1]);
          if (next) commit(&sfull[t]);
          else if (k >= 0 && k + 1 == own) commit(&pvdone[t]);
          if (k >= 0 && k < own) commit(&vempty[s]);
          if (next) {
            commit(&kempty[ka]);
            if (fresh) commit(&kempty[kb]);
            kc += fresh ? 2 : 1;
            if (DUP) kc += jn + 1 >= jfresh ? 2 : 1;
          }
          if (k + 2 == own || (own == 0 && k < 0)) commit(qempty);  // no later S reads Q
          j = jn;
        }
        J += n;
        Jt += own;
        K += n + max(n - jfresh, 0);
      }
    }
  } else if (warp < 8) {
    const int tid = threadIdx.x - 128;
    bool ok = true;
    int J = 0;
    Piece p;
    for (int w = w0; ok && next_piece(a, plan, from, w, w1, p);) {
      for (int j = 0; j < p.tiles(); ++j, ++J) {
        const int s = J % kNV, par = (J / kNV) & 1;
        if (!(ok = wait(&cfull[s], par, status, abort))) break;
        if (!p.fresh(j)) {
          if (!(ok = wait(&vempty[s], par ^ 1, status, abort))) break;
          const uint8_t* src = smem + Smem::oVc + s * Smem::kK;
          uint8_t* dst = smem + Smem::oVf + s * Smem::kF16;
          const int valid = p.len - (p.t0 + j) * kTK;
#pragma unroll
          for (int it = 0; it < HD / 16; ++it) {
            const int id = it * 128 + tid, row = id / (HD / 16), c = id % (HD / 16);
            uint4 v = *reinterpret_cast<const uint4*>(src + row * HD + ((c ^ swz<HD>(row)) << 4));
            if (row >= valid) v = make_uint4(0, 0, 0, 0);  // what lies behind the sequence never enters an MMA
            uint4 h[2];
            e4m3x4_f16x4(v.x, h[0].x, h[0].y);
            e4m3x4_f16x4(v.y, h[0].z, h[0].w);
            e4m3x4_f16x4(v.z, h[1].x, h[1].y);
            e4m3x4_f16x4(v.w, h[1].z, h[1].w);
            uint8_t* d = dst + (c / 4) * Smem::kBox + row * 128;
            const int ch = (c % 4) * 2, f = c / 4;  // the two boxes' lanes store their halves in opposite order: no bank conflicts
            *reinterpret_cast<uint4*>(d + (((ch + f) ^ (row & 7)) << 4)) = f ? h[1] : h[0];
            *reinterpret_cast<uint4*>(d + (((ch + 1 - f) ^ (row & 7)) << 4)) = f ? h[0] : h[1];
          }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&cempty[s]);
          mbar_arrive(&vfull[s]);
        }
      }
    }
  } else {
    const int t = (warp - 8) / 4, q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + lane_base + 128 * t, tO = tmem + lane_base + kColO + 128 * t;
    bool ok = true;
    int Jt = 0, np = 0, met = 0;  // own tiles, pieces that had some, phases of meet
    float2* ml = reinterpret_cast<float2*>(smem + Smem::oMl);
    auto join = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      const bool all = wait(meet, met++ & 1, status, abort);
      tc_fence_after();
      return all;
    };
    Piece p;
    for (int w = w0; ok && next_piece(a, plan, from, w, w1, p);) {
      const int n = DUP ? (p.tiles() + 1 - t) / 2 : p.tiles(), bh = p.b * a.Hkv + p.hk;
      const int rpart = DUP ? r : 128 * t + r, ridx = p.row0 + rpart;
      auto tile = [&](int k) { return DUP ? 2 * k + t : k; };  // own tile k
      const bool valid_row = ridx < grp_rows;
      const int qx = valid_row ? pp.qexp[(size_t)bh * grp_rows + ridx] : 0;
      const int qi = valid_row ? ridx % a.C : 0;
      // exponents of the tile's two blocks: key 0, key 1, value 0, value 1
      auto exps = [&](int j, int (&e)[4]) {
        const bool fresh = p.fresh(j);
        const int i = (p.t0 + j - (fresh ? p.ntc : 0)) * 2, nb = fresh ? pp.Cp / kKv8Block : a.nblk;
        const uint8_t* ke = (fresh ? pp.kexp : a.Ke) + (size_t)bh * nb;
        const uint8_t* ve = (fresh ? pp.vexp : a.Ve) + (size_t)bh * nb;
        const int i1 = min(i + 1, nb - 1);
        e[0] = ke[i];
        e[1] = ke[i1];
        e[2] = ve[i];
        e[3] = ve[i1];
      };
      int ex[4], en[4] = {};
      if (n > 0) exps(tile(0), en);
      float m_run = -INFINITY, l_run = 0.f;
      int ve_top = kKv8Emin;  // checked here: by the four warps of the V codes it cost 3 % more
      for (int own = 0; own < n; ++own) {
        const int j = tile(own);
#pragma unroll
        for (int k = 0; k < 4; ++k) ex[k] = en[k] - kKv8Bias;
        if (own + 1 < n) exps(tile(own + 1), en);
        if (!(ok = wait(&sfull[t], (Jt + own) & 1, status, abort))) break;
        tc_fence_after();
        const bool fresh = p.fresh(j);
        const int key0 = (p.t0 + j - (fresh ? p.ntc : 0)) * kTK;
        int lim = (fresh ? a.C : p.len) - key0;  // columns of the tile that this row sees
        ve_top = max(ve_top, lim > kKv8Block ? max(ex[2], ex[3]) : ex[2]);
        if (fresh && a.causal) lim = min(lim, qi - key0 + 1);
        // Two passes over the scores, 64 columns (one block's scales) at a
        // time: kept in registers between them they would need twice the
        // registers and unrolled code that no instruction cache holds.
        auto load = [&](int b, float (&s)[64]) {
          tmem_ld32_async(tS + 64 * b, *reinterpret_cast<float(*)[32]>(s));
          tmem_ld32_async(tS + 64 * b + 32, *reinterpret_cast<float(*)[32]>(s + 32));
          tmem_wait_ld();
        };
        if (__any_sync(0xffffffffu, lim < kTK)) {
          // a sequence's last tile, or a causal one: masked in TMEM, so that the
          // passes' loops hold no code for it (prompt pieces 41.6 -> 39.8 us)
#pragma unroll 1
          for (int c = 0; c < kTK; c += 16) {
            uint32_t s[16];
            tmem_ld16(tS + c, s);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (c + e >= lim) s[e] = __float_as_uint(-INFINITY);
            tmem_st16(tS + c, s);
          }
          tmem_wait_st();
        }
        float mx = -INFINITY;
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
          float s[64];
          load(b, s);
          float x0 = fmaxf(s[0], s[1]), x1 = fmaxf(s[2], s[3]), x2 = fmaxf(s[4], s[5]), x3 = fmaxf(s[6], s[7]);
#pragma unroll
          for (int c = 8; c < 64; c += 8) {
            x0 = fmax3(x0, s[c], s[c + 1]);
            x1 = fmax3(x1, s[c + 2], s[c + 3]);
            x2 = fmax3(x2, s[c + 4], s[c + 5]);
            x3 = fmax3(x3, s[c + 6], s[c + 7]);
          }
          const int ke = b ? ex[1] : ex[0], ve = b ? ex[3] : ex[2];
          mx = fmaxf(mx, fmaf(fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)), scale_log2 * pow2i(qx + ke), (float)ve));
        }
        if (own == 0) {
          m_run = mx;
        } else {
          const bool need = mx > m_run + kLazy;
          if (__any_sync(0xffffffffu, need)) {
            const float corr = need ? ex2_approx(m_run - mx) : 1.0f;
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(tO + 16 * c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tmem_st16(tO + 16 * c, o);
            }
            if (need) {
              l_run *= corr;
              m_run = mx;
            }
          }
        }
        const float mm = m_run == -INFINITY ? 0.f : m_run - kHeadroom;
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {  // 32 columns of P each
          float s[64];
          load(b, s);
          const int ke = b ? ex[1] : ex[0], ve = b ? ex[3] : ex[2];
          const float c = scale_log2 * pow2i(qx + ke), off = (float)ve - mm;
          const uint64_t c2 = f2_pack(c, c), off2 = f2_pack(off, off);
          uint64_t rs[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t hw[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float t0, t1;
              f2_unpack(f2_fma(f2_pack(s[32 * h + 2 * e], s[32 * h + 2 * e + 1]), c2, off2), t0, t1);
              const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
              rs[e & 1] = f2_add(rs[e & 1], f2_pack(p0, p1));
              hw[e] = pack_f16(p0, p1);
            }
            tmem_st16(tS + 32 * b + 16 * h, hw);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pready[2 * t + b]);
          float x0, x1;
          f2_unpack(f2_add(rs[0], rs[1]), x0, x1);
          l_run = fmaf(x0 + x1, pow2i(-ve), l_run);
        }
      }
      if (!ok || (n > 0 && !(ok = wait(&pvdone[t], np & 1, status, abort)))) break;
      tc_fence_after();
      if (ve_top > kKv8EmaxAttn) atomicExch(status, kStatusValue);
      const bool whole = p.t0 == 0 && p.t1 == p.nt;
      const size_t slot = ((size_t)blockIdx.x * 2 + (p.t0 > 0 ? 0 : 1)) * (DUP ? 2 : 1) + (DUP ? t : 0);
      const float inv = l_run == 0.f ? 0.f : 1.0f / l_run;
      __nv_bfloat16* orow = valid_row ? kv8_out_row(a, p.b, p.hk, ridx) : nullptr;
      if (DUP && whole) {
        // half of the columns each, from both row tiles' outputs
        ml[128 * t + r] = make_float2(m_run, l_run);
        if (!(ok = join())) break;
        const float2 m0 = ml[r], m1 = ml[128 + r];
        const float M = fmaxf(m0.x, m1.x);
        float w0 = m0.x == -INFINITY ? 0.f : exp2f(m0.x - M), w1 = m1.x == -INFINITY ? 0.f : exp2f(m1.x - M);
        const float l = fmaf(w0, m0.y, w1 * m1.y), scale = l == 0.f ? 0.f : 1.0f / l;
        w0 *= scale;
        w1 *= scale;
#pragma unroll 1
        for (int c = HD / 64 * t; c < HD / 64 * (t + 1); ++c) {
          float o[32], o1[32];
          tmem_ld32(tmem + lane_base + kColO + 32 * c, o);
          tmem_ld32(tmem + lane_base + kColO + 128 + 32 * c, o1);
#pragma unroll
          for (int e = 0; e < 32; ++e)  // with one tile TMEM holds another piece's output in the second place
            o[e] = p.tiles() > 1 ? fmaf(w0, o[e], w1 * o1[e]) : w0 * o[e];
          if (!valid_row) continue;
          uint4* dst = reinterpret_cast<uint4*>(orow + 32 * c);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            dst[q] = make_uint4(pack_bf16(o[8 * q], o[8 * q + 1]), pack_bf16(o[8 * q + 2], o[8 * q + 3]),
                                pack_bf16(o[8 * q + 4], o[8 * q + 5]), pack_bf16(o[8 * q + 6], o[8 * q + 7]));
        }
        if (!(ok = join())) break;  // both have read the outputs, and ml
        Jt += n;
        np += n > 0;
        continue;
      }
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        float o[32];
        tmem_ld32(tO + 32 * c, o);
        if (n == 0) {  // no tile for this row tile: TMEM holds another piece's output
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (!valid_row) continue;
        if (!DUP && whole) {
          uint4* dst = reinterpret_cast<uint4*>(orow + 32 * c);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            dst[q] = make_uint4(pack_bf16(o[8 * q] * inv, o[8 * q + 1] * inv), pack_bf16(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                                pack_bf16(o[8 * q + 4] * inv, o[8 * q + 5] * inv), pack_bf16(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *kv8_part(a, slot, 8 * c + q, rpart) = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          if (c == 0)
            a.ml[slot * a.prows + rpart] = make_float2(m_run, l_run);
        }
      }
      Jt += n;
      np += n > 0;
    }
  }
  __syncthreads();
  if (*abort) {  // copies in flight land before the CTA's shared memory goes
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- prep --
// q to two E4M3 terms and a scale per row (8 elements a lane);
// new keys to two E4M3 terms and new values to f16, with a scale per 64 tokens
// (one CTA per block, zeros behind the last token).
template <int HD>
__global__ void __launch_bounds__(256) kv8_prep_kernel(Kv8AttnArgs a, Kv8Prep pp, int kv_ctas) {
  constexpr int LPR = HD / 8, RPC = 256 / LPR;  // lanes per row, rows per CTA
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= kv_ctas) {
    const long long row = (long long)(blockIdx.x - kv_ctas) * RPC + tid / LPR;
    const bool there = row < pp.qrows;
    const uint4 w = there ? *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + row * HD +
                                                            (tid % LPR) * 8)
                          : make_uint4(0, 0, 0, 0);
    unsigned top = abs_top(w);
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = top_exponent(top);
    float x[8];
    unpack8(w, pow2i(-e), x);
    uint2 hi, lo;
    split8(x, hi, lo);
    if (!there) return;
    *reinterpret_cast<uint2*>(pp.qterms + row * HD + (tid % LPR) * 8) = hi;
    *reinterpret_cast<uint2*>(pp.qterms + ((size_t)pp.qrows + row) * HD + (tid % LPR) * 8) = lo;
    if (tid % LPR == 0) pp.qexp[row] = e;
    return;
  }
  __shared__ unsigned red[8];
  const int nb = pp.Cp / kKv8Block, isv = blockIdx.x & 1, blk = (blockIdx.x >> 1) % nb, bh = (blockIdx.x >> 1) / nb;
  const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(isv ? a.vn : a.kn) + (size_t)bh * a.C * HD;
  uint4 w[kKv8Block / RPC];
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < kKv8Block / RPC; ++i) {
    const int row = blk * kKv8Block + i * RPC + tid / LPR;
    w[i] = row < a.C ? *reinterpret_cast<const uint4*>(src + (size_t)row * HD + (tid % LPR) * 8) : make_uint4(0, 0, 0, 0);
    top = __vmaxu2(top, abs_top(w[i]));
  }
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  if (tid % 32 == 0) red[tid / 32] = top;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, red[tid % 8]);
  const int e = top_exponent(top);
  if (tid == 0) (isv ? pp.vexp : pp.kexp)[(size_t)bh * nb + blk] = (uint8_t)(e + kKv8Bias);
#pragma unroll
  for (int i = 0; i < kKv8Block / RPC; ++i) {
    const size_t row = (size_t)bh * pp.Cp + blk * kKv8Block + i * RPC + tid / LPR;
    float x[8];
    unpack8(w[i], pow2i(-e), x);
    if (isv) {
      *reinterpret_cast<uint4*>(pp.vf16 + row * HD * 2 + (tid % LPR) * 16) =
          make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]), pack_f16(x[6], x[7]));
    } else {
      uint2 hi, lo;
      split8(x, hi, lo);
      *reinterpret_cast<uint2*>(pp.kterms + row * HD + (tid % LPR) * 8) = hi;
      *reinterpret_cast<uint2*>(pp.kterms + ((size_t)pp.krows + row) * HD + (tid % LPR) * 8) = lo;
    }
  }
}

}  // namespace

template <int HD, bool DUP>
static cudaError_t run_tc(const Kv8AttnArgs& a, const Kv8Prep& pp, cudaStream_t st) {
  constexpr auto kern = kv8_attn_tc_kernel<HD, DUP>;
  const uint64_t cached = (uint64_t)a.B * a.Hkv * a.cap;
  CUtensorMap mQ, mK, mV, mKn, mVn;
  if (!make_tmap_2d(&mQ, pp.qterms, HD, 2 * (uint64_t)pp.qrows, HD, HD, 128, true, HD) ||
      !make_tmap_2d(&mK, a.K, HD, cached, HD, HD, kTK, true, HD) ||
      !make_tmap_2d(&mV, a.V, HD, cached, HD, HD, kTK, true, HD))
    return cudaErrorInvalidValue;
  mKn = mK;  // without new tokens neither is used
  mVn = mV;
  if (a.kn && (!make_tmap_2d(&mKn, pp.kterms, HD, 2 * (uint64_t)pp.krows, HD, HD, kTK, true, HD) ||
               !make_tmap_2d(&mVn, pp.vf16, HD, (uint64_t)pp.krows, HD * 2, 64, kTK)))
    return cudaErrorInvalidValue;
  cudaError_t e = set_smem_once<kern>(Smem<HD>::kTotal);
  if (e != cudaSuccess) return e;
  const int kv_ctas = a.kn ? 2 * a.B * a.Hkv * (pp.Cp / kKv8Block) : 0;
  e = launch_pdl(kv8_prep_kernel<HD>, dim3(kv_ctas + cdiv(pp.qrows, 256 / (HD / 8))), dim3(256), 0, st, a, pp, kv_ctas);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(kKv8Ctas), dim3(kThreads), Smem<HD>::kTotal, st, mQ, mK, mV, mKn, mVn, a, pp,
                    1.4426950408889634f / sqrtf((float)HD));
}

cudaError_t launch_kv8_attention_tc(const Kv8AttnArgs& a, const Kv8Prep& pp, cudaStream_t st) {
  if (a.hd == 64) return a.subs == 2 ? run_tc<64, true>(a, pp, st) : run_tc<64, false>(a, pp, st);
  if (a.hd == 128) return a.subs == 2 ? run_tc<128, true>(a, pp, st) : run_tc<128, false>(a, pp, st);
  return cudaErrorInvalidValue;
}

}  // namespace dg

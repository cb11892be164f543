// Tensor-core (tcgen05 + TMA) attention over the 8-bit prefix cache for many
// query rows per kv head (canvases and prompt pieces), head dims 64 and 128.
//
// A CTA owns 256 query rows (two tiles of 128) of one (sequence, kv head) and a
// run of 128-key tiles; the tiles of a call are dealt to the CTAs in equal
// shares (dg_kv8.cuh), parts are merged by kv8_merge_kernel.  What the 8-bit
// cache changes against the bf16 kernel (dg_attn_tc.cu):
//  - Eight warps expand the codes on their way to shared memory, keys with their
//    block's scale to bf16 and values to f16, both exactly.  Queries and the new
//    tokens' keys enter as the bf16 they are, so a score is the fp32 sum of exact
//    products, whatever else is in its row, its block or behind its mask.  (Queries
//    and new keys as two E4M3 terms each, against the codes as they lie, spared the
//    expansion: 117 us where this takes 124.  But they took 2^-18 of the largest element
//    of the row, or of 64 tokens, from every other: one padded token's key could
//    cost the others all their bits.)
//  - P V of cached tiles runs in f16: p' is rounded to f16 (2^-11), once, where
//    bf16 would need two terms.  New tokens' values keep their exponent range:
//    bf16 products, p' split into two bf16 (2^-17), both over the 32 keys' own scores.
//  - Value scales never touch the codes: 2^ve joins the exponent of the probability
//    (the running maximum is that of s + ve), whose share of the row sum is taken
//    back.
//
// Warp roles (20 warps, one CTA per SM):
//   warp 0       TMA: queries per piece
//   warps 1, 2   MMA, one for each row tile, taking turns: P_t V of key tile j, then
//                S_t of tile j + 1, so that one row tile's softmax and waits run
//                under the other's products
//   warps 4-7    values: codes to f16, new rows copied
//   warps 8-15   softmax, one thread per row, 64 columns at a time (up to 128 rows 32,
//                for shorter code); P over S in TMEM
//   warps 16-19  keys: codes to bf16, new rows copied
//
// Measured: a canvas of 256 rows over 131072 rows of 8 heads 124 us (the two
// products at the measured bf16 rate: 72), 1.11 PFLOP/s; a key tile takes some 3700
// cycles, 2048 of them MMAs.  A row tile's chain (scores ready, two passes of
// softmax 2100 to 2400 cycles, P V and the next S 1500) bounds it, lengthened by
// what the expansion takes of the issue slots, of shared memory (MMA operands,
// codes and expanded tiles: some 2500 cycles a tile) and of the instruction
// cache, where what the warps run at a time has to fit: with the expansion unrolled,
// and the loop over the probabilities choosing between cached and new tiles, it ran
// 128 us, calls of many short units a third longer.  Tried and slower: rings of code
// tiles filled by TMA, 161 us (with half tiles) and 143 (for keys or values alone),
// prefetches into L2 132 to 137, eight warps to each tile 142, four in all 162.
// Tried and slower while the codes entered the MMA as they lie (117 us then): two
// threads a row (24 warps of 80 registers, 123 us; 20 of 96, 168 us), the
// scores read once block by block (123 to 129), the probabilities made on the old
// maximum in one pass and again where it grew (135), loads 32 columns ahead (129),
// scores of 64 keys at a time, two of them in flight to a row tile (126 to 129:
// the softmax no longer waits, but an MMA of 64 columns takes as long as one of
// 128 and the MMA warps have twice the turns), MMA warps without turns (143).
// Head dim 64 has half the MMAs and the same softmax: 256 rows over 32768 rows of
// 8 heads 35 us (the warp-MMA kernel 92.7).
#include <cfloat>

#include "dg_kv8.cuh"

namespace dg {
namespace {

constexpr int kTK = 128;                   // keys per tile
constexpr int kThreads = 640;
// Registers: the block is launched with 96 a thread; the softmax warps take 120,
// the others keep 80.  The shares add up to no more than the launch's, or a
// setmaxnreg would wait for ever.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 120, kOtherRegs = 80;
static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs, "registers of one block");
constexpr int kNS = 2;                     // slots of expanded keys, and of values
constexpr float kHeadroom = 8.0f;          // p' of a row's maximum is 2^8 ..
constexpr float kLazy = 6.0f;              // .. to 2^14: O is rescaled when the maximum grew by more than 2^6

template <int HD>
struct Smem {
  static constexpr int kBox = kTK * 128;             // 64 16-bit columns of a tile
  static constexpr int kTile = HD / 64 * kBox;       // a tile of 128 rows in 16 bits
  static constexpr int oK = 2 * kTile;               // behind the queries of both row tiles
  static constexpr int oV = oK + kNS * kTile;
  static constexpr int kCode = kTK * HD;             // codes on their way: a tile of keys, one of values
  static constexpr int oC = oV + kNS * kTile;
  static constexpr int oBar = oC + 2 * kCode;
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
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
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
// Shared-memory descriptors (swizzle over rows of 128 bytes, 1024 between 8-row
// groups) as a low word, address and leading offset, and a high word.
DG_DEV uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3FFFFu) >> 4) | (lbo >> 4 << 16); }
DG_DEV uint64_t desc64(uint32_t lo) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "n"(hi));
  return d;
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

DG_DEV uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
DG_DEV uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 16 codes to 16-bit words: keys times f as bf16, values as f16 (exact).
DG_DEV void expand_keys(const uint4& w, float f, uint4 (&h)[2]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
  const uint64_t f2 = f2_pack(f, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t x[2];
    e4m3x4_f16x4(u[j], x[0], x[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&x[k]));
      float y0, y1;
      f2_unpack(f2_mul(f2_pack(t.x, t.y), f2), y0, y1);
      o[2 * j + k] = pack_bf16(y0, y1);
    }
  }
  h[0] = make_uint4(o[0], o[1], o[2], o[3]);
  h[1] = make_uint4(o[4], o[5], o[6], o[7]);
}
DG_DEV void expand_values(const uint4& w, uint4 (&h)[2]) {
  e4m3x4_f16x4(w.x, h[0].x, h[0].y);
  e4m3x4_f16x4(w.y, h[0].z, h[0].w);
  e4m3x4_f16x4(w.z, h[1].x, h[1].y);
  e4m3x4_f16x4(w.w, h[1].z, h[1].w);
}

// The part of four warps: the tiles of all of the CTA's pieces, keys or values, to
// the MMA's buffer of kNS slots.  A thread takes 16-byte chunks of codes and has the
// next tile's on their way while it expands this one's, in slots of its own in shared
// memory.  The loop is rolled: alone a key tile takes 528 cycles unrolled, but
// beside the softmax's code no instruction cache held it, and it took 2700 (375
// ragged sequences of up to 2000 rows, 4 heads of 24 rows: 296 us, with codes in
// registers, as unrolled loops allow; 207 rolled).
template <int HD, bool KEYS>
DG_DEV void expand_tiles(const Kv8AttnArgs& a, const Kv8Plan& plan, int2& from, int w0, int w1, uint8_t* buf, uint64_t* full,
                         uint64_t* empty, uint8_t* slots, volatile int* abort) {
  using Smem = Smem<HD>;
  constexpr int IT = HD / 16, RS = 128 / IT;  // chunks of a row, and of a thread, whose rows are RS apart
  static_assert(RS % 8 == 0, "one swizzle a thread");
  // A row's chunk c of 16 elements is chunks 2 c and 2 c + 1 of its 16-bit row in box
  // c / 4.  Eight consecutive lanes take four chunks of one box of two rows, whose
  // swizzles make up the other four 16-byte banks.
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const int r0 = HD == 128 ? tid / 32 * 4 + lane / 16 * 2 + (lane >> 2 & 1) : tid / 4;
  const int c = HD == 128 ? (lane & 3) + (lane >> 3 & 1) * 4 : tid % 4;
  const int o0 = c / 4 * Smem::kBox + r0 * 128 + ((c % 4 * 2 ^ (r0 & 7)) << 4), o1 = o0 ^ 16;
  const uint8_t *codes = KEYS ? a.K : a.V, *rows = reinterpret_cast<const uint8_t*>(KEYS ? a.kn : a.vn);
  slots += tid * 16;  // chunk `it` of this thread at 2048 it
  bool ok = true;
  int J = 0;
  Piece p;
  for (int w = w0; ok && next_piece(a, plan, from, w, w1, p);) {
    const int n = p.tiles(), cached = min(p.t1, p.ntc) - p.t0;
    const size_t bh = (size_t)p.b * a.Hkv + p.hk;
    const uint8_t *src = codes + (bh * a.cap + (size_t)p.t0 * kTK + r0) * HD + c * 16, *Ke = a.Ke + bh * a.nblk;
    int left = p.len - p.t0 * kTK - r0, blk = p.t0 * 2, ke0 = 0, ke1 = 0;
    // chunk `it` of the tile at src on its way; what lies behind the sequence is not read
    auto load = [&](int it) {
      const bool there = it * RS < left;
      cp_async16(slots + it * 2048, there ? src + it * RS * HD : codes, there);
    };
    auto scales = [&]() {
      ke0 = Ke[blk];
      ke1 = Ke[min(blk + 1, a.nblk - 1)];
    };
    if (KEYS && cached > 0) scales();
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (cached > 0) load(it);
      cp_async_commit();  // a group for each chunk
    }
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const int s = (J + j) & 1, par = ((J + j) >> 1) & 1;
      if (!(ok = wait(&empty[s], par ^ 1, a.status, abort))) break;
      uint8_t* dst = buf + s * Smem::kTile;
      auto store = [&](int it, const uint4 (&h)[2]) {
        *reinterpret_cast<uint4*>(dst + o0 + it * RS * 128) = h[0];
        *reinterpret_cast<uint4*>(dst + o1 + it * RS * 128) = h[1];
      };
      if (j < cached) {
        const bool more = j + 1 < cached;
        const float f0 = pow2i(ke0 - kKv8Bias), f1 = pow2i(ke1 - kKv8Bias);
        blk += 2;
        if (KEYS && more) scales();
        src += kTK * HD;
        left -= kTK;
        cp_async_wait<IT - 1>();
        uint4 next = *reinterpret_cast<const uint4*>(slots);
#pragma unroll 1
        for (int it = 0; it < IT; ++it) {  // the first half of the chunks are the tile's first block
          const uint4 x = next;
          cp_async_wait<IT - 2>();
          next = *reinterpret_cast<const uint4*>(slots + (it + 1 < IT ? it + 1 : 0) * 2048);  // (behind the last: not used)
          uint4 h[2];
          if (KEYS) expand_keys(x, it < IT / 2 ? f0 : f1, h);
          else expand_values(x, h);
          store(it, h);
          if (more) load(it);  // the chunk's slot again: its values have been used
          cp_async_commit();
        }
      } else {
        // new rows as they are, zeros behind the last; the values' magnitudes are looked at
        const int key0 = (p.t0 + j - p.ntc) * kTK;
        const uint8_t* nr = rows + ((bh * a.C + key0 + r0) * HD + c * 16) * 2;
        const int nleft = a.C - key0 - r0;
        unsigned top = 0;
#pragma unroll 4
        for (int it = 0; it < IT; ++it) {
          uint4 h[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
          if (it * RS < nleft) {
            h[0] = load16(nr + it * RS * HD * 2);
            h[1] = load16(nr + it * RS * HD * 2 + 16);
          }
          if (!KEYS) top = __vmaxu2(top, __vmaxu2(abs_top(h[0]), abs_top(h[1])));
          store(it, h);
        }
        if (!KEYS && top_exponent(max(top & 0xffffu, top >> 16)) > kKv8EmaxAttn) atomicExch(a.status, kStatusValue);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
    }
    J += n;
  }
}

// DUP: up to 128 query rows.  Both row tiles hold the same rows and row tile t
// takes key tiles t, t + 2, ..; their outputs are two parts, which the softmax
// warps join themselves where the CTA has all of the unit's tiles.
template <int HD, bool DUP>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_attn_tc_kernel(const __grid_constant__ CUtensorMap mQ, Kv8AttnArgs a, float scale_log2) {
  using Smem = Smem<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {  // uniform over the CTA: return before any barrier
    if (threadIdx.x == 0) atomicExch(a.status, kStatusTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::oBar);
  uint64_t* qfull = bars;
  uint64_t* qempty = qfull + 1;
  uint64_t* kfull = qempty + 1;      // [kNS] keys ready for the MMA
  uint64_t* kempty = kfull + kNS;    // [kNS]
  uint64_t* vfull = kempty + kNS;    // [kNS] values
  uint64_t* vempty = vfull + kNS;    // [kNS]
  uint64_t* sfull = vempty + kNS;    // [2]
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
    for (int s = 0; s < kNS; ++s) {
      mbar_init(&kfull[s], 4);
      mbar_init(&kempty[s], readers);
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 0) {
      if (blockIdx.x == 0)
        for (int b = lane; b < a.B; b += 32)
          if (a.len[b] < 0 || a.len[b] > a.cap) atomicExch(status, kStatusCapacity);
      if (lane == 0) tma_prefetch(&mQ);
      bool ok = true;
      int np = 0;
      Piece p;
      for (int w = w0; ok && next_piece(a, plan, from, w, w1, p); ++np) {
        if (lane == 0) {
          ok = mbar_wait(qempty, (np & 1) ^ 1, status, abort);
          if (ok) {
            const int qrow = (p.b * a.Hkv + p.hk) * grp_rows + p.row0;
            mbar_arrive_expect_tx(qfull, 2 * Smem::kTile);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int x = 0; x < HD / 64; ++x)
                tma_load_2d(smem + t * Smem::kTile + x * Smem::kBox, &mQ, qfull, 64 * x, qrow + (DUP ? 0 : 128 * t));
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
    } else if (warp < 3) {
      const int t = warp - 1;
      constexpr uint32_t idS = idesc_bf16(128, kTK, false);
      constexpr uint32_t idPV = idesc_f16(128, HD, true), idPVn = idesc_bf16(128, HD, true);
      const uint32_t lo_q = desc_lo(smem_u32(smem + t * Smem::kTile), 16), lo_k = desc_lo(smem_u32(smem + Smem::oK), 16);
      const uint32_t lo_v = desc_lo(smem_u32(smem + Smem::oV), Smem::kBox);
      const uint32_t tS = tmem + 128 * t, tO = tmem + kColO + 128 * t;
      bool ok = true;
      static_assert(kNS == 2, "slots from running counts");
      int J = 0, Jt = 0, np = 0, turns = t ^ 1;  // tiles, own tiles, pieces so far; parity of the turn
      const int stride = DUP ? 2 : 1, begin = DUP ? t : 0;
      Piece p;
      for (int w = w0; ok && next_piece(a, plan, from, w, w1, p); ++np) {
        const int n = p.tiles(), jfresh = max(p.ntc - p.t0, 0);  // tiles from jfresh on hold new tokens
        const int own = DUP ? (n + 1 - t) >> 1 : n, steps = DUP ? (n + 1) >> 1 : n;
        int j = begin - stride;                           // own key tile k of the piece
        ok = wait(qfull, np & 1, status, abort);
        // Step k: P_t V of own key tile k, then S_t of own tile k + 1.  The two warps
        // take turns, step by step, which keeps the row tiles' softmax phases apart
        // (left alone they fall into step, and the tensor core idles while both
        // wait); each does its waiting and committing during the other's turn.
        // A commit covers all MMAs of its thread before it, so S_t of tile k + 1
        // also says that P_t V of tile k is done.
#pragma unroll 1
        for (int k = -1; k < steps && ok; ++k) {
          const int s = (J + j) & 1, jn = j + stride, sn = (J + jn) & 1;
          const bool next = k + 1 < own;
          if (next && !(ok = wait(&kfull[sn], ((J + jn) >> 1) & 1, status, abort))) break;
          if (k >= 0 && k < own) {
            if (!(ok = wait(&vfull[s], ((J + j) >> 1) & 1, status, abort))) break;
            // (the first P of a piece also says that the last one's output has been read)
            if (!(ok = wait(&pready[2 * t], (Jt + k) & 1, status, abort))) break;
            if (!(ok = wait(&turn[t], turns, status, abort))) break;
            tc_fence_after();
            const uint32_t v = lo_v + s * (Smem::kTile >> 4);
            const bool fresh = j >= jfresh;
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
              if (b) {
                if (!(ok = wait(&pready[2 * t + 1], (Jt + k) & 1, status, abort))) break;
                tc_fence_after();
              }
              const uint32_t vb = v + b * (64 * 128 >> 4);
              if (!fresh) {
#pragma unroll
                for (int k4 = 0; k4 < 4; ++k4)
                  mma_pv(tO, tS + 32 * b + 8 * k4, desc64(vb + k4 * (2048 >> 4)), idPV, (k | b | k4) ? 1u : 0u);
              } else {  // both terms of P
#pragma unroll
                for (int k4 = 0; k4 < 8; ++k4)  // of each 32 keys the first terms, then the second
                  mma_pv(tO, tS + 64 * b + 8 * k4, desc64(vb + (k4 / 4 * 2 + (k4 & 1)) * (2048 >> 4)), idPVn, (k | b | k4) ? 1u : 0u);
              }
            }
            if (!ok) break;
          } else {
            if (!(ok = wait(&turn[t], turns, status, abort))) break;
            tc_fence_after();
          }
          turns ^= 1;
          if (next) {
            const uint32_t kd = lo_k + sn * (Smem::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint32_t o = (kk >> 2) * (Smem::kBox >> 4) + 2 * (kk & 3);
              mma_s(tS, desc64(lo_q + o), desc64(kd + o), idS, kk ? 1u : 0u);
            }
          }
          if (lane == 0) mbar_arrive(&turn[t ^ 1]);
          if (next) commit(&sfull[t]);
          else if (k >= 0 && k + 1 == own) commit(&pvdone[t]);
          if (k >= 0 && k < own) commit(&vempty[s]);
          if (next) commit(&kempty[sn]);
          if (k + 2 == own || (own == 0 && k < 0)) commit(qempty);  // no later S reads Q
          j = jn;
        }
        J += n;
        Jt += own;
      }
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    expand_tiles<HD, false>(a, plan, from, w0, w1, smem + Smem::oV, vfull, vempty, smem + Smem::oC + Smem::kCode, abort);
  } else if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    expand_tiles<HD, true>(a, plan, from, w0, w1, smem + Smem::oK, kfull, kempty, smem + Smem::oC, abort);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = (warp - 8) / 4, q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + lane_base + 128 * t, tO = tmem + lane_base + kColO + 128 * t;
    constexpr int NC = DUP ? 32 : 64;  // columns of scores at a time
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
      const int qi = valid_row ? ridx % a.C : 0;
      // value exponents of the tile's two blocks; new tokens have none
      const uint8_t* Ve = a.Ve + (size_t)bh * a.nblk;
      auto exps = [&](int j, int (&e)[2]) {
        e[0] = e[1] = kKv8Bias;
        if (p.fresh(j)) return;
        const int i = (p.t0 + j) * 2;
        e[0] = Ve[i];
        e[1] = Ve[min(i + 1, a.nblk - 1)];
      };
      int ex[2], en[2] = {};
      if (n > 0) exps(tile(0), en);
      float m_run = -INFINITY, l_run = 0.f;
      int ve_top = kKv8Emin;  // checked here: by the four warps of the V codes it cost 3 % more
      for (int own = 0; own < n; ++own) {
        const int j = tile(own);
#pragma unroll
        for (int k = 0; k < 2; ++k) ex[k] = en[k] - kKv8Bias;
        if (own + 1 < n) exps(tile(own + 1), en);
        if (!(ok = wait(&sfull[t], (Jt + own) & 1, status, abort))) break;
        tc_fence_after();
        const bool fresh = p.fresh(j);
        const int key0 = (p.t0 + j - (fresh ? p.ntc : 0)) * kTK;
        int lim = (fresh ? a.C : p.len) - key0;  // columns of the tile that this row sees
        ve_top = max(ve_top, lim > kKv8Block ? max(ex[0], ex[1]) : ex[0]);
        if (fresh && a.causal) lim = min(lim, qi - key0 + 1);
        // Two passes over the scores, NC columns (of one block's scales) at a
        // time: kept in registers between them they would need twice the
        // registers and unrolled code that no instruction cache holds.
        auto load = [&](int q, float (&s)[NC]) {
#pragma unroll
          for (int i = 0; i < NC / 32; ++i) tmem_ld32_async(tS + NC * q + 32 * i, *reinterpret_cast<float(*)[32]>(s + 32 * i));
          tmem_wait_ld();
        };
        if (__any_sync(0xffffffffu, lim < kTK)) {
          // a sequence's last tile, or a causal one: masked in TMEM, so that the
          // passes' loops hold no code for it (in them it cost prompt pieces 4 %)
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
        for (int q = 0; q < kTK / NC; ++q) {
          float s[NC];
          load(q, s);
          float x0 = fmaxf(s[0], s[1]), x1 = fmaxf(s[2], s[3]), x2 = fmaxf(s[4], s[5]), x3 = fmaxf(s[6], s[7]);
#pragma unroll
          for (int c = 8; c < NC; c += 8) {
            x0 = fmax3(x0, s[c], s[c + 1]);
            x1 = fmax3(x1, s[c + 2], s[c + 3]);
            x2 = fmax3(x2, s[c + 4], s[c + 5]);
            x3 = fmax3(x3, s[c + 6], s[c + 7]);
          }
          mx = fmaxf(mx, fmaf(fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)), scale_log2, (float)(NC * q < kKv8Block ? ex[0] : ex[1])));
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
        const uint64_t c2 = f2_pack(scale_log2, scale_log2);
        auto ready = [&](int half) {  // this half of the tile's P is in TMEM
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pready[2 * t + half]);
        };
        // apart, so that the loop of the cached tiles is short
        if (!fresh) {
#pragma unroll 1
          for (int q = 0; q < kTK / NC; ++q) {  // half as many columns of P each
            float s[NC];
            load(q, s);
            const int ve = NC * q < kKv8Block ? ex[0] : ex[1];
            const float off = (float)ve - mm;
            const uint64_t off2 = f2_pack(off, off);
            uint64_t rs[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
            for (int h = 0; h < NC / 32; ++h) {
              uint32_t hw[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float t0, t1;
                f2_unpack(f2_fma(f2_pack(s[32 * h + 2 * e], s[32 * h + 2 * e + 1]), c2, off2), t0, t1);
                const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
                rs[e & 1] = f2_add(rs[e & 1], f2_pack(p0, p1));
                hw[e] = pack_f16(p0, p1);
              }
              tmem_st16(tS + NC / 2 * q + 16 * h, hw);
            }
            if (NC == 64 || (q & 1)) ready(NC * q / kKv8Block);
            float x0, x1;
            f2_unpack(f2_add(rs[0], rs[1]), x0, x1);
            l_run = fmaf(x0 + x1, pow2i(-ve), l_run);
          }
        } else {
          const uint64_t off2 = f2_pack(-mm, -mm);
#pragma unroll 1
          for (int q = 0; q < kTK / 32; ++q) {  // both terms of P over its own scores
            float s[32];
            tmem_ld32(tS + 32 * q, s);
            uint64_t rs[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float t0, t1;
              f2_unpack(f2_fma(f2_pack(s[2 * e], s[2 * e + 1]), c2, off2), t0, t1);
              const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
              rs[e & 1] = f2_add(rs[e & 1], f2_pack(p0, p1));
              hi[e] = pack_bf16(p0, p1);
              lo[e] = pack_bf16(p0 - __uint_as_float(hi[e] << 16), p1 - __uint_as_float(hi[e] & 0xffff0000u));
            }
            tmem_st16(tS + 32 * q, hi);
            tmem_st16(tS + 32 * q + 16, lo);
            if (q & 1) ready(q >> 1);
            float x0, x1;
            f2_unpack(f2_add(rs[0], rs[1]), x0, x1);
            l_run += x0 + x1;
          }
        }
      }
      if (!ok || (n > 0 && !(ok = wait(&pvdone[t], np & 1, status, abort)))) break;
      tc_fence_after();
      if (ve_top > kKv8EmaxAttn || (valid_row && kv8_far(m_run))) atomicExch(status, kStatusValue);
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
          if (valid_row) {
            uint4* dst = reinterpret_cast<uint4*>(orow + 32 * c);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              dst[q] = make_uint4(pack_bf16(o[8 * q], o[8 * q + 1]), pack_bf16(o[8 * q + 2], o[8 * q + 3]),
                                  pack_bf16(o[8 * q + 4], o[8 * q + 5]), pack_bf16(o[8 * q + 6], o[8 * q + 7]));
          }
          __syncwarp();  // the next TMEM load is the whole warp's
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
        if (valid_row && !DUP && whole) {
          uint4* dst = reinterpret_cast<uint4*>(orow + 32 * c);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            dst[q] = make_uint4(pack_bf16(o[8 * q] * inv, o[8 * q + 1] * inv), pack_bf16(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                                pack_bf16(o[8 * q + 4] * inv, o[8 * q + 5] * inv), pack_bf16(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
        } else if (valid_row) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *kv8_part(a, slot, 8 * c + q, rpart) = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          if (c == 0) a.ml[slot * a.prows + rpart] = make_float2(m_run, l_run);
        }
        __syncwarp();
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

}  // namespace

template <int HD, bool DUP>
static cudaError_t run_tc(const Kv8AttnArgs& a, cudaStream_t st) {
  constexpr auto kern = kv8_attn_tc_kernel<HD, DUP>;
  CUtensorMap mQ;
  if (!make_tmap_2d(&mQ, a.q, HD, (uint64_t)a.B * a.Hq * a.C, HD * 2, 64, 128)) return cudaErrorInvalidValue;
  static const cudaError_t regs = [] {  // what the register shares are reckoned from
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kern);
    return e == cudaSuccess && fa.numRegs < kLaunchRegs ? cudaErrorLaunchOutOfResources : e;
  }();
  if (regs != cudaSuccess) return regs;
  cudaError_t e = set_smem_once<kern>(Smem<HD>::kTotal);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(kKv8Ctas), dim3(kThreads), Smem<HD>::kTotal, st, mQ, a,
                    1.4426950408889634f / sqrtf((float)HD));
}

cudaError_t launch_kv8_attention_tc(const Kv8AttnArgs& a, cudaStream_t st) {
  if (a.hd == 64) return a.subs == 2 ? run_tc<64, true>(a, st) : run_tc<64, false>(a, st);
  if (a.hd == 128) return a.subs == 2 ? run_tc<128, true>(a, st) : run_tc<128, false>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace dg

// decode_vs.cu -- split-K paged MLA decode over an e4m3 cache with group
// scales, for row tiles of up to 128 query rows: a cluster of two CTAs that
// split the value columns (sm_103a).
//
// The fp32 accumulator of 128 rows x 512 value columns fills a whole tensor
// memory, so a row tile takes two SMs. Here each CTA owns all 128 rows and 256
// of the value columns; both compute all scores and the same softmax. That
// doubles Q K^T, but no probabilities cross between the SMs (distributed
// shared memory moves about 20 bytes a clock), the softmax has its row in one
// thread with no exchange but one of maxima, and the second-largest cost, the
// epilogue, is halved. Per 128 keys a CTA issues
//   S[rows, keys]  = Q K^T   M = 128 rows, N = 128 keys, K = 576: A = q from
//                            TMEM (512 latent dims) and shared memory (64 rope
//                            dims), B = the key rows of the ring, K-major:
//                            18 kind::f8f6f4 instructions of 64 cycles;
//   O[rows, 256]  += P V     M = 128 rows, N = 256 columns, K = 128 keys, P as
//                            two e4m3 terms (hi, lo), V = the same key rows
//                            read MN-major: 8 instructions of 128 cycles.
// That is 2176 tensor cycles per 128 keys, close to what the shared memory's
// 128 bytes a clock allow for the operands, the copies in and P (284 KB, 2220
// cycles). The softmax of 128 x 128 scores takes the eight warps about 1300
// issue cycles and runs beside them: S is read into registers at once, so
// that the next chunk's Q K^T can overwrite it while its weights are formed,
// and one buffer of S and one of P are enough.
//
// Every key box is read from memory once, by one CTA of the cluster, and
// multicast to the ring slot of both (dense); a slot is refilled once both
// CTAs have released it, a box of the other half's value columns after Q K^T,
// one of the own half after P V. Sparse lists gather their rows with TMA
// gather4, each CTA for itself.
//
// Weights: with group scales the thread's scores become t = score + log2 s and
// the weights 2^(t - m) multiply the codes (KeyScale). They are formed as
// p = 2^(t - m_ref + 4) with a reference that moves only when a chunk maximum
// exceeds it by more than 4 (O is then rescaled in TMEM), so p <= 2^8 fits
// e4m3 and hi + lo carry 8 bits of it.
//
// Warps: 0, 2, 12, 13 load, 1 issues Q K^T, 3 P V, 4-11 softmax and epilogue
// (a TMEM lane quarter of the rows and a half of the keys each). Every wait is
// bounded: a timeout records a code in the status word, stops the CTA's work,
// drains what was issued and exits.
#include <atomic>
#include <climits>

#include "common.cuh"
#include "internal.h"
#include "tc_ops.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace tc;

constexpr int kRows = 128;               // query rows of a tile: M
constexpr int kKeys = 128;               // keys per chunk: N of Q K^T, K of P V
constexpr int kHalf = 64;                // keys per TMA box, and per softmax warp
constexpr int kSlot = kKeys * 128;       // ring slot: a 128-byte column box of a chunk (or of q)
constexpr int kRSlot = kKeys * 64;       // rope ring slot
constexpr int kBoxes = 5;                // per chunk: 4 latent boxes and the rope box
constexpr int kSlots = 10;               // even: the two value boxes of a CTA are neighbours
constexpr int kRSlots = 2;
constexpr int kQStage = kSlots - 4;      // q's latent boxes land in the last four slots
constexpr int kThreads = 448;
constexpr int kProducers = 4;            // warps 0, 2, 12, 13
constexpr int kSoftWarps = 8;            // warps 4-11
constexpr int kPTile = kRows * kHalf;    // one e4m3 term of P for 64 keys
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;           // 256 columns
constexpr uint32_t kTmemS = 256;         // 128
constexpr uint32_t kTmemQ = 384;         // 128: 512 latent dims, four to a column
constexpr uint64_t kDefaultWaitNs = 2000000000ull;
constexpr uint32_t kSleepNs = 20000;
constexpr float kPBias = 4.f;            // p = 2^(t - m_ref + kPBias) <= 2^(2 kPBias)
constexpr float kMove = 4.f;             // m_ref moves when a chunk max exceeds it by more

enum : int {
  kFull = 0,                 // [kSlots] ring slot loaded
  kEmpty = kSlots,           // [kSlots] ring slot released (by every CTA that loads into it)
  kRFull = 2 * kSlots,       // [kRSlots]
  kREmpty = kRFull + kRSlots,
  kQFull = kREmpty + kRSlots,  // q staged
  kQTmem,                    // q copied to TMEM: the staging slots are free
  kSFull,                    // S written
  kSFree,                    // S read
  kPFull,                    // P written
  kPFree,                    // P V complete: P may be replaced, O holds the chunk
  kX,                        // [4] the two warps of a row quarter have posted
  kDrain = kX + 4,           // the Q K^T issuer's MMAs complete
  kDrainPV,
  kNumBars
};

// Shared memory: header, q's rope columns, P, the rope ring, the ring.
constexpr int kOffBar = 0;
constexpr int kOffTslot = 384;
constexpr int kOffAbort = 388;
constexpr int kOffIssued = 448;           // [kSlots + kRSlots] int: last use issued per slot
constexpr int kOffXMax = 1024;            // [2][2][128] chunk maxima by parity and key half
constexpr int kOffLsum = 3072;            // [2][128] row sums by key half
constexpr int kOffScale = 4096;           // [8 warps][mul, add, inv][64]
constexpr int kOffQR = 10240;             // 128 rows x 64 bytes, 64-byte swizzle
constexpr int kOffP = kOffQR + kRSlot;    // [key half][hi, lo] tiles, 64-byte swizzle
constexpr int kOffRope = kOffP + 4 * kPTile;
constexpr int kOffRing = kOffRope + kRSlots * kRSlot;
constexpr int kSmem = kOffRing + kSlots * kSlot + 1024;  // + alignment slack
static_assert(kNumBars * 8 <= kOffTslot && kOffIssued + 4 * (kSlots + kRSlots) <= kOffXMax, "header space");
static_assert(kOffScale + kSoftWarps * 3 * kHalf * 4 <= kOffQR, "scale space");
static_assert(kSlots % 2 == 0 && kSlots >= 8 && kSmem <= 232448, "shared memory budget");

struct VsMaps {
  CUtensorMap q;     // q as [T*H rows, 576] e4m3, box 128 bytes x 128 rows
  CUtensorMap qr;    // the same, box 64 bytes (the rope columns)
  CUtensorMap kv;    // cache as [NB*BS rows, 576], box 128 bytes x 64 rows; sparse: x 1 row
  CUtensorMap kvr;   // the same, box 64 bytes
  CUtensorMap out;   // out as [T*H, 1, 512] bf16, box 32 rows x 64 columns, 128-byte swizzle
  CUtensorMap part;  // partials as [slot rows, 1, 512] or [T*H, NS, 512] fp32, box 32 x 32
};

struct Ctx {
  uint8_t* smem;
  uint32_t bar0;
  volatile int* abort;
  int* status;
  uint64_t limit_ns;
  uint32_t tbase;
  int tid, warp, lane, rank;
  int H, unit, tok0, qlen, row0, rows_total, part_len;
  int64_t list_base;
  int seg, seg_start, seg_end, n_chunks;
  int pslot;  // partial slot of a balanced piece, -1: write out/lse
  bool fin;
  __device__ uint32_t bar(int i) const { return bar0 + 8u * i; }
};

__device__ __forceinline__ void report(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// Bounded wait on a barrier phase, sleeping; false on timeout (recorded) or
// abort. kCluster: acquire at cluster scope (barriers the peer arrives on).
template <bool kCluster = false>
__device__ bool wait_phase(const Ctx& x, uint32_t bar, uint32_t parity, int code) {
  if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  const uint32_t nap = x.limit_ns < kSleepNs ? static_cast<uint32_t>(x.limit_ns) : kSleepNs;
  while (!(kCluster ? mbar_try_wait_cluster_sleep(bar, parity, nap) : mbar_try_wait_sleep(bar, parity, nap))) {
    if (*x.abort) return false;
    if (global_timer_ns() - t0 > x.limit_ns) {
      report(x.status, code);
      *x.abort = 1;
      return false;
    }
  }
  return true;
}
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(const Ctx& x, uint32_t bar, uint32_t parity, int code) {
  return __all_sync(0xffffffffu, wait_phase<kCluster>(x, bar, parity, code)) != 0;
}
// Wait that ignores the abort flag (teardown), still bounded.
__device__ void drain_wait(const Ctx& x, uint32_t bar, uint32_t parity, int code) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_cluster_sleep(bar, parity, kSleepNs)) {
    if (global_timer_ns() - t0 > kDefaultWaitNs) {
      report(x.status, code);
      return;
    }
  }
}

// Release of a ring slot by this CTA's MMAs: to both CTAs where both fill it.
template <bool SPARSE>
__device__ __forceinline__ void release(uint32_t bar) {
  if constexpr (SPARSE)
    mma_commit(bar);
  else
    mma_commit_mc(bar, static_cast<uint16_t>(3));
}

// Cache slot of key position pos (-1 past the segment or for an unused list entry).
template <bool SPARSE>
__device__ __forceinline__ int key_slot(const Ctx& x, const DecodeParams& p, const int32_t* bt_row, int pos) {
  if (pos >= x.seg_end) return -1;
  if constexpr (SPARSE) return p.slots[x.list_base + pos];
  const int blk = pos / p.block_size;
  return bt_row[blk] * p.block_size + (pos - blk * p.block_size);
}

// ------------------------------------------------------------------ producers
// Box j of chunk g: latent box j < 4 goes to ring slot i % kSlots, i = 4 g + j,
// the rope box to rope slot g % kRSlots. The first use of the slots that
// stage q waits until both CTAs have copied q out.
__device__ __forceinline__ bool slot_ready(const Ctx& x, bool rope, int slot, int use, bool cluster) {
  if (use >= 1) {
    const uint32_t b = x.bar(rope ? kREmpty + slot : kEmpty + slot);
    return cluster ? wait_phase<true>(x, b, (use - 1) & 1, 11) : wait_phase<false>(x, b, (use - 1) & 1, 11);
  }
  return rope || slot < kQStage || wait_phase<true>(x, x.bar(kQTmem), 0, 10);
}

// Dense: box b = 5 g + j is loaded by CTA b % 2, there by producer warp
// (b / 2) % 4, and multicast to both. The whole warp looks up the cache rows
// of 16 chunks at a time, a window ahead; lane 0 issues.
__device__ void produce_dense(const Ctx& x, const VsMaps& maps, const DecodeParams& p, int pidx) {
  const int lane = x.lane;
  volatile int* issued = reinterpret_cast<volatile int*>(x.smem + kOffIssued);
  if (lane == 0) {
    tma_prefetch_desc(&maps.kv);
    tma_prefetch_desc(&maps.kvr);
  }
  const uint64_t pol = l2_evict_first();  // each key row is read once
  const int32_t* bt_row = p.block_table + static_cast<int64_t>(x.unit) * p.bt_stride;
  auto lookup = [&](int w0) {  // cache row of this lane's (chunk, half) in the window at w0
    const int s = key_slot<false>(x, p, bt_row, x.seg_start + (w0 + (lane >> 1)) * kKeys + (lane & 1) * kHalf);
    return s < 0 ? 0 : s;
  };
  int cur = lookup(0), nxt = lookup(16);
  bool ok = true;
  for (int g = 0; g < x.n_chunks && ok; ++g) {
    if (g > 0 && (g & 15) == 0) {
      cur = nxt;
      nxt = lookup(g + 16);
    }
    const int row0 = __shfl_sync(0xffffffffu, cur, 2 * (g & 15));
    const int row1 = __shfl_sync(0xffffffffu, cur, 2 * (g & 15) + 1);
    const bool two = x.seg_start + g * kKeys + kHalf < x.seg_end;
    if (lane == 0) {
      for (int j = 0; j < kBoxes; ++j) {
        const int b = g * kBoxes + j;
        if ((b & 1) != x.rank || ((b >> 1) % kProducers) != pidx) continue;
        const bool rope = j == kBoxes - 1;
        const int i = rope ? g : 4 * g + j;
        const int slot = i % (rope ? kRSlots : kSlots);
        const int use = i / (rope ? kRSlots : kSlots);
        if (!slot_ready(x, rope, slot, use, true)) {
          ok = false;
          break;
        }
        const int box = rope ? kRSlot : kSlot;
        const uint32_t bytes = two ? box : box / 2;
        const uint32_t full = x.bar(rope ? kRFull + slot : kFull + slot);
        mbar_arrive_expect_tx(full, bytes);
        // the peer's phase of this slot also waits for the box
        mbar_arrive_expect_tx_cluster(map_to_rank(full, x.rank ^ 1), bytes);
        const uint32_t dst = smem_u32(x.smem + (rope ? kOffRope + slot * kRSlot : kOffRing + slot * kSlot));
        const CUtensorMap* map = rope ? &maps.kvr : &maps.kv;
        tma_load_2d_mc_hint(dst, map, 128 * j, row0, full, 3, pol);
        if (two) tma_load_2d_mc_hint(dst + box / 2, map, 128 * j, row1, full, 3, pol);
        atomicMax(const_cast<int*>(issued + (rope ? kSlots + slot : slot)), use);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  }
  __syncwarp();
}

// Sparse: box 5 g + j is gathered by warp (5 g + j) % 4 of each CTA: lane l
// issues one gather4 of the rows of keys 4 l .. 4 l + 3. A key without a slot
// reads row 0: its score is masked and its value row zeroed by the softmax
// warps, whatever the row holds.
__device__ void produce_sparse(const Ctx& x, const VsMaps& maps, const DecodeParams& p, int pidx) {
  const int lane = x.lane;
  volatile int* issued = reinterpret_cast<volatile int*>(x.smem + kOffIssued);
  if (lane == 0) {
    tma_prefetch_desc(&maps.kv);
    tma_prefetch_desc(&maps.kvr);
  }
  const uint64_t pol = l2_evict_first();
  int nx[4];
  auto lookup = [&](int g) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      nx[k] = g < x.n_chunks ? key_slot<true>(x, p, nullptr, x.seg_start + g * kKeys + 4 * lane + k) : 0;
  };
  lookup(0);
  bool ok = true;
  for (int g = 0; g < x.n_chunks && ok; ++g) {
    int r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = nx[k] >= 0 ? nx[k] : 0;
    lookup(g + 1);
    for (int j = 0; j < kBoxes && ok; ++j) {
      if ((g * kBoxes + j) % kProducers != pidx) continue;
      const bool rope = j == kBoxes - 1;
      const int i = rope ? g : 4 * g + j;
      const int slot = i % (rope ? kRSlots : kSlots);
      const int use = i / (rope ? kRSlots : kSlots);
      ok = __all_sync(0xffffffffu, slot_ready(x, rope, slot, use, false)) != 0;
      if (!ok) break;
      const uint32_t full = x.bar(rope ? kRFull + slot : kFull + slot);
      if (lane == 0) {
        mbar_arrive_expect_tx(full, rope ? kRSlot : kSlot);
        atomicMax(const_cast<int*>(issued + (rope ? kSlots + slot : slot)), use);
      }
      __syncwarp();
      if (rope)
        tma_gather4_hint(smem_u32(x.smem + kOffRope + slot * kRSlot + 256 * lane), &maps.kvr, 128 * j, r[0], r[1], r[2],
                         r[3], full, pol);
      else
        tma_gather4_hint(smem_u32(x.smem + kOffRing + slot * kSlot + 512 * lane), &maps.kv, 128 * j, r[0], r[1], r[2],
                         r[3], full, pol);
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ MMA issue
template <bool SPARSE>
__device__ void qk_issue(const Ctx& x, const VsMaps& maps) {
  if (x.lane != 0 || x.n_chunks == 0) return;
  constexpr uint32_t kId = instr_desc(kRows, kKeys, 0, 0, false, false);
  const uint64_t k_desc = smem_desc_sw128(smem_u32(x.smem + kOffRing), 16, 1024);
  const uint64_t r_desc = smem_desc_sw64(smem_u32(x.smem + kOffRope), 512);
  const uint64_t q_desc = smem_desc_sw64(smem_u32(x.smem + kOffQR), 512);
  tma_prefetch_desc(&maps.q);
  mbar_arrive_expect_tx(x.bar(kQFull), 4 * kSlot + kRSlot);
  const int qrow = x.tok0 * x.H + x.row0;
  for (int j = 0; j < 4; ++j)
    tma_load_2d(smem_u32(x.smem + kOffRing + (kQStage + j) * kSlot), &maps.q, 128 * j, qrow, x.bar(kQFull));
  tma_load_2d(smem_u32(x.smem + kOffQR), &maps.qr, 512, qrow, x.bar(kQFull));
  bool ok = wait_phase(x, x.bar(kQFull), 0, 20) && wait_phase<true>(x, x.bar(kQTmem), 0, 21);
  const uint32_t d = x.tbase + kTmemS;
  for (int g = 0; g < x.n_chunks && ok; ++g) {
    if (g >= 1 && !wait_phase(x, x.bar(kSFree), (g - 1) & 1, 22)) break;
#pragma unroll
    for (int j = 0; j < kBoxes; ++j) {
      const bool rope = j == kBoxes - 1;
      const int i = rope ? g : 4 * g + j;
      const int slot = i % (rope ? kRSlots : kSlots);
      const int use = i / (rope ? kRSlots : kSlots);
      if (!wait_phase<!SPARSE>(x, x.bar(rope ? kRFull + slot : kFull + slot), use & 1, 23)) {
        ok = false;
        break;
      }
      fence_after_sync();
      if (rope) {
        const uint64_t b = r_desc + static_cast<uint64_t>(slot * (kRSlot >> 4));
#pragma unroll
        for (int s = 0; s < 2; ++s) mma_ss_f8(d, q_desc + 2 * s, b + 2 * s, kId, 1u);
        release<SPARSE>(x.bar(kREmpty + slot));
      } else {
        const uint64_t b = k_desc + static_cast<uint64_t>(slot * (kSlot >> 4));
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_ts_f8(d, x.tbase + kTmemQ + 32 * j + 8 * s, b + 2 * s, kId, (j | s) != 0 ? 1u : 0u);
        if ((j >> 1) != x.rank) release<SPARSE>(x.bar(kEmpty + slot));  // its values are the peer's
      }
    }
    if (!ok) break;
    mma_commit(x.bar(kSFull));
  }
  mma_commit(x.bar(kDrain));
  drain_wait(x, x.bar(kDrain), 0, 25);
}

template <bool SPARSE>
__device__ void pv_issue(const Ctx& x) {
  if (x.lane != 0 || x.n_chunks == 0) return;
  constexpr uint32_t kId = instr_desc(kRows, 256, 0, 0, false, true);
  const uint64_t v_desc = smem_desc_sw128(smem_u32(x.smem + kOffRing), kSlot, 1024);  // MN-major
  const uint64_t p_desc = smem_desc_sw64(smem_u32(x.smem + kOffP), 512);
  const uint32_t d = x.tbase + kTmemO;
  for (int g = 0; g < x.n_chunks; ++g) {
    // P written; the softmax waited for S, whose Q K^T waited for these boxes
    if (!wait_phase(x, x.bar(kPFull), g & 1, 24)) break;
    fence_after_sync();
    const int slot = (4 * g + 2 * x.rank) % kSlots;
    const uint64_t vb = v_desc + static_cast<uint64_t>(slot * (kSlot >> 4));
    const bool two = x.seg_start + g * kKeys + kHalf < x.seg_end;  // else the second half holds no key
#pragma unroll
    for (int ks = 0; ks < kKeys / 32; ++ks) {
      if (ks >= 2 && !two) break;
      const uint64_t av = p_desc + static_cast<uint64_t>(((ks >> 1) * 2 * kPTile + (ks & 1) * 32) >> 4);
      const uint64_t bv = vb + static_cast<uint64_t>((ks * 32 * 128) >> 4);
      mma_ss_f8(d, av, bv, kId, (g | ks) != 0 ? 1u : 0u);
      mma_ss_f8(d, av + static_cast<uint64_t>(kPTile >> 4), bv, kId, 1u);
    }
    release<SPARSE>(x.bar(kEmpty + slot));
    release<SPARSE>(x.bar(kEmpty + slot + 1));
    mma_commit(x.bar(kPFree));
  }
  mma_commit(x.bar(kDrainPV));
  drain_wait(x, x.bar(kDrainPV), 0, 26);
}

// ------------------------------------------------------------------ softmax + epilogue
template <bool SPARSE>
__device__ void softmax_rows(const Ctx& x, const VsMaps& maps, const DecodeParams& p) {
  const int lane = x.lane;
  const int sw = x.warp - 4;
  const int q4 = x.warp & 3;               // TMEM lane quarter of this warp
  const int h = sw >> 2;                   // its half of a chunk's keys, and of the CTA's value columns
  const int r = q4 * 32 + lane;            // row within the tile
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const int H = x.H;
  const int rho = x.row0 + r;
  const bool row_ok = rho < x.rows_total;
  const int vis = !row_ok ? 0 : (SPARSE ? INT_MAX : x.part_len - x.qlen + rho / H + 1);
  const float scale2 = p.score_scale_log2;
  bool ok = true;

  // this row of q, staged in the ring's last slots, into TMEM (two of the
  // four latent boxes each)
  if (x.n_chunks > 0) {
    ok = warp_wait(x, x.bar(kQFull), 0, 30);
    if (ok) {
#pragma unroll 1
      for (int j = 2 * h; j < 2 * h + 2; ++j) {
        const uint8_t* src = x.smem + kOffRing + (kQStage + j) * kSlot + r * 128;
        uint32_t v[32];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint4 t = *reinterpret_cast<const uint4*>(src + ((q ^ (r & 7)) << 4));
          v[4 * q] = t.x;
          v[4 * q + 1] = t.y;
          v[4 * q + 2] = t.z;
          v[4 * q + 3] = t.w;
        }
        tmem_st_32x32b_x32(x.tbase + lane_off + kTmemQ + 32 * j, v);
      }
      tmem_st_wait();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(x.bar(kQTmem));
        mbar_arrive_cluster(map_to_rank(x.bar(kQTmem), x.rank ^ 1));
      }
    }
  }

  float* xmax = reinterpret_cast<float*>(x.smem + kOffXMax);
  float* lsum = reinterpret_cast<float*>(x.smem + kOffLsum);
  float* ksc = reinterpret_cast<float*>(x.smem + kOffScale) + sw * 3 * kHalf;
  uint8_t* prow = x.smem + kOffP + h * 2 * kPTile + r * 64;
  const int pswz = (r >> 1) & 3;           // 64-byte swizzle of the row's 16-byte chunks
  // slots of the warp's keys (lane l: keys l and l + 32 of its half) two
  // chunks ahead and their scales one ahead, so that no read is waited for
  const int32_t* bt_row = SPARSE ? nullptr : p.block_table + static_cast<int64_t>(x.unit) * p.bt_stride;
  auto slot_of = [&](int g, int i) {
    return g < x.n_chunks ? key_slot<SPARSE>(x, p, bt_row, x.seg_start + g * kKeys + h * kHalf + lane + 32 * i) : -1;
  };
  auto scale_of = [&](int slot) {
    return slot >= 0 ? p.kv_scales[static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.scale_group)] : 1.f;
  };
  int sl0 = slot_of(0, 0), sl1 = slot_of(0, 1);
  float sc0 = scale_of(sl0), sc1 = scale_of(sl1);
  int nsl0 = slot_of(1, 0), nsl1 = slot_of(1, 1);

  float m_ref = -INFINITY, m_true = -INFINITY, l = 0.f;
  for (int g = 0; g < x.n_chunks && ok; ++g) {
    const uint64_t kmask = static_cast<uint64_t>(__ballot_sync(0xffffffffu, sl0 >= 0)) |
                           (static_cast<uint64_t>(__ballot_sync(0xffffffffu, sl1 >= 0)) << 32);
    {
      const KeyScale k0 = key_scale(sc0, scale2), k1 = key_scale(sc1, scale2);
      __syncwarp();  // every lane is done with the previous chunk's scales
      ksc[lane] = k0.mul;
      ksc[lane + 32] = k1.mul;
      ksc[kHalf + lane] = k0.add;
      ksc[kHalf + lane + 32] = k1.add;
      ksc[2 * kHalf + lane] = k0.inv;
      ksc[2 * kHalf + lane + 32] = k1.inv;
      sl0 = nsl0;
      sl1 = nsl1;
      sc0 = scale_of(sl0);
      sc1 = scale_of(sl1);
      nsl0 = slot_of(g + 2, 0);
      nsl1 = slot_of(g + 2, 1);
      __syncwarp();
    }
    ok = warp_wait(x, x.bar(kSFull), g & 1, 31);
    if (!ok) break;
    fence_after_sync();
    float s[64];
    {
      uint32_t sr[64];
      tmem_ld_32x32b_x64(x.tbase + lane_off + kTmemS + kHalf * h, sr);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 64; ++j) s[j] = __uint_as_float(sr[j]);
    }
    fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kSFree));  // the next chunk's Q K^T may overwrite S
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
      const float4 mu = *reinterpret_cast<const float4*>(ksc + j);
      const float4 ad = *reinterpret_cast<const float4*>(ksc + kHalf + j);
      s[j] = fmaf(s[j], mu.x, ad.x);
      s[j + 1] = fmaf(s[j + 1], mu.y, ad.y);
      s[j + 2] = fmaf(s[j + 2], mu.z, ad.z);
      s[j + 3] = fmaf(s[j + 3], mu.w, ad.w);
    }
    // keys that exist and that the row may see
    const int lim = min(vis, x.seg_end) - (x.seg_start + g * kKeys + h * kHalf);
    if (lim < kHalf || kmask != ~0ull) {
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (!(j < lim && ((kmask >> j) & 1ull))) s[j] = -INFINITY;
    }
    float m8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m8[i] = s[i];
#pragma unroll
    for (int j = 8; j < 64; ++j) m8[j & 7] = fmaxf(m8[j & 7], s[j]);
    const float mine = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                             fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
    // the row's maximum over both key halves
    float* xm = xmax + (g & 1) * 2 * kRows;
    xm[h * kRows + r] = mine;
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kX + q4));
    ok = warp_wait(x, x.bar(kX + q4), g & 1, 32);
    if (!ok) break;
    const float mx = fmaxf(mine, xm[(h ^ 1) * kRows + r]);
    m_true = fmaxf(m_true, mx);
    float alpha = 1.f;
    if (mx > m_ref + kMove) {  // also when the row's first visible key arrives
      if (m_ref != -INFINITY) {
        alpha = fast_exp2(m_ref - mx);
        l *= alpha;
      }
      m_ref = mx;
    }
    // p as hi + lo e4m3 terms, 16 keys to a 16-byte chunk of each tile
    const float base = m_ref == -INFINITY ? 0.f : m_ref - kPBias;
    uint32_t hi[16], lo[16];
    float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float4 iv = *reinterpret_cast<const float4*>(ksc + 2 * kHalf + 4 * j);
      const float p0 = fast_exp2(s[4 * j] - base), p1 = fast_exp2(s[4 * j + 1] - base);
      const float p2 = fast_exp2(s[4 * j + 2] - base), p3 = fast_exp2(s[4 * j + 3] - base);
      ps[0] = fmaf(p0, iv.x, ps[0]);
      ps[1] = fmaf(p1, iv.y, ps[1]);
      ps[2] = fmaf(p2, iv.z, ps[2]);
      ps[3] = fmaf(p3, iv.w, ps[3]);
      uint32_t h0, h1, l0, l1;
      p_terms(p0, p1, h0, l0);
      p_terms(p2, p3, h1, l1);
      hi[j] = h0 | (h1 << 16);
      lo[j] = l0 | (l1 << 16);
    }
    l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
    // the previous chunk's P V has read P and O is complete up to it
    if (g >= 1) {
      ok = warp_wait(x, x.bar(kPFree), (g - 1) & 1, 33);
      if (!ok) break;
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
        // some rows moved their reference: this warp rescales its rows of its
        // half of the value columns
        fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const uint32_t ta = x.tbase + lane_off + kTmemO + 128 * h + 32 * c;
          uint32_t o[32];
          tmem_ld_32x32b_x32(ta, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st_32x32b_x32(ta, o);
        }
        tmem_st_wait();
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      *reinterpret_cast<uint4*>(prow + ((c ^ pswz) << 4)) = make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
      *reinterpret_cast<uint4*>(prow + kPTile + ((c ^ pswz) << 4)) =
          make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
    }
    // value rows of keys that do not exist (stale or unloaded ring contents,
    // cache rows past the sequence, unused list entries) must not reach O
    // through p = 0: they are zeroed, a quarter by each warp of the half
    if (kmask != ~0ull && (h == 0 || x.seg_start + g * kKeys + kHalf < x.seg_end)) {
      const int slot = (4 * g + 2 * x.rank) % kSlots;
      uint8_t* box = x.smem + kOffRing + (slot + ((lane >> 3) & 1)) * kSlot + h * kHalf * 128 + (lane & 7) * 16;
      for (int j = q4 + 4 * (lane >> 4); j < kHalf; j += 8)
        if (!((kmask >> j) & 1ull)) *reinterpret_cast<uint4*>(box + j * 128) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kPFull));
  }

  // ---------------------------------------------------------------- epilogue
  if (ok) {
    lsum[h * kRows + r] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kX + q4));
    ok = warp_wait(x, x.bar(kX + q4), x.n_chunks & 1, 34);
  }
  if (ok && x.n_chunks > 0) {
    ok = warp_wait(x, x.bar(kPFree), (x.n_chunks - 1) & 1, 35);
    fence_after_sync();
  }
  if (!ok) return;
  float mult = 0.f;
  if (row_ok) {
    const float L = lsum[r] + lsum[kRows + r];
    const float base = m_ref == -INFINITY ? 0.f : m_ref - kPBias;  // the sums' reference
    const int head = rho % H;
    const int64_t th = static_cast<int64_t>(x.tok0 + rho / H) * H + head;
    const bool writes = x.rank == 0 && h == 0;
    if (x.fin) {
      float lse = -INFINITY;
      if (p.sinks != nullptr) {
        const float s2 = p.sinks[head] * kLog2e;
        const float M = fmaxf(L > 0.f ? base : -INFINITY, s2);
        const float e = L > 0.f ? exp2f(base - M) : 0.f;
        const float W = L * e + exp2f(s2 - M);
        mult = e / W;
        lse = kLn2 * (M + log2f(W));
      } else if (L > 0.f) {
        mult = 1.f / L;
        lse = kLn2 * (base + log2f(L));
      }
      if (writes) p.lse[th] = lse;
    } else {
      mult = L > 0.f ? 1.f / L : 0.f;
      if (writes) {
        const int64_t ts = x.pslot >= 0 ? static_cast<int64_t>(x.pslot) * p.slot_rows + r : th * p.num_segments + x.seg;
        p.segm_max[ts] = L > 0.f ? m_true : -INFINITY;
        p.segm_expsum[ts] = L > 0.f ? L * exp2f(base - m_true) : 0.f;
      }
    }
  }
  // Each warp scales its 32 rows x 128 columns and stages them, 128 bytes of
  // each row at a time, in the 128-byte swizzle, in the ring (which holds no
  // more boxes in use). When all 32 rows are valid one TMA tensor store writes
  // each staged tile (two in flight); otherwise every store instruction covers
  // four 128-byte row pieces. (TMEM loads are warp-collective.)
  const int col0 = 256 * x.rank + 128 * h;
  const int wr = x.row0 + 32 * q4;          // the warp's first row within the unit
  if (wr >= x.rows_total) return;
  const bool whole = wr + 32 <= x.rows_total;
  const int z0 = x.fin || x.pslot < 0 ? x.tok0 * H + wr : x.pslot * p.slot_rows + 32 * q4;
  const int y0 = x.fin || x.pslot >= 0 ? 0 : x.seg;
  const CUtensorMap* map = x.fin ? &maps.out : &maps.part;
  uint8_t* stage = x.smem + kOffRing + sw * 8192;
  const int qc = lane & 7;                  // 16-byte piece of a 128-byte row piece
  int staged = 0;
  auto store = [&](const uint32_t (&w)[32], int col) {
    uint8_t* buf = stage + (staged & 1) * 4096;
    if (whole && staged >= 2 && lane == 0) bulk_wait_read<1>();  // the store that read this buffer
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q)
      *reinterpret_cast<uint4*>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    if (whole) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(map, smem_u32(buf), col, y0, z0);
        bulk_commit_group();
      }
    } else {
      __syncwarp();
#pragma unroll 1
      for (int it = 0; it < 8; ++it) {
        const int row = 4 * it + (lane >> 3);
        const int rr = wr + row;
        if (rr >= x.rows_total) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(buf + row * 128 + ((qc ^ (row & 7)) << 4));
        const int64_t th = static_cast<int64_t>(x.tok0 + rr / H) * H + rr % H;
        const int64_t ts = x.pslot >= 0 ? static_cast<int64_t>(x.pslot) * p.slot_rows + (rr - x.row0)
                                        : th * p.num_segments + x.seg;
        uint8_t* dst = x.fin ? static_cast<uint8_t*>(p.out) + (th * kRank + col) * 2
                             : reinterpret_cast<uint8_t*>(p.segm_out + ts * kRank + col);
        *reinterpret_cast<uint4*>(dst + qc * 16) = v;
      }
      __syncwarp();
    }
    ++staged;
  };
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t o[64];
    if (x.n_chunks > 0) {
      tmem_ld_32x32b_x64(x.tbase + lane_off + kTmemO + 128 * h + 64 * c, o);
      tmem_ld_wait();
    } else {
#pragma unroll
      for (int j = 0; j < 64; ++j) o[j] = 0u;
    }
    uint32_t w[32];
    if (x.fin) {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * mult, __uint_as_float(o[2 * j + 1]) * mult);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      store(w, col0 + 64 * c);
    } else {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(o[32 * hf + j]) * mult);
        store(w, col0 + 64 * c + 32 * hf);
      }
    }
  }
  if (lane == 0) bulk_wait_all();  // tiles read and written before the CTA exits
  __syncwarp();
}

template <bool SPARSE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    decode_vs_kernel(const __grid_constant__ VsMaps maps, const DecodeParams p, int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctx x;
  x.smem = smem;
  x.status = status;
  x.limit_ns = p.wait_ns != 0 ? p.wait_ns : kDefaultWaitNs;
  x.tid = threadIdx.x;
  x.warp = x.tid >> 5;
  x.lane = x.tid & 31;
  x.rank = static_cast<int>(cluster_ctarank());
  int tile, item_begin = 0, item_end = 0;
  x.pslot = -1;
  if (p.items != nullptr) {
    // balanced schedule: both CTAs read the same item, once the grid that
    // wrote the list has completed; the merge may launch once every CTA has started
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int item = blockIdx.x >> 1;
    if (item >= *p.n_items) return;
    const int4 a = reinterpret_cast<const int4*>(p.items)[2 * item];
    const int4 b = reinterpret_cast<const int4*>(p.items)[2 * item + 1];
    x.unit = a.x;
    tile = a.y;
    item_begin = a.z;
    item_end = a.w;
    x.pslot = b.x;
    x.seg = 0;
    x.fin = x.pslot < 0;
  } else {
    tile = blockIdx.x >> 1;
    x.seg = blockIdx.y;
    x.unit = blockIdx.z;
    x.fin = p.final_mode != 0;
  }
  x.H = p.num_heads;
  x.qlen = 1;
  x.tok0 = x.unit;
  x.list_base = 0;
  if constexpr (SPARSE) {
    if (p.slot_indptr != nullptr) {
      x.list_base = p.slot_indptr[x.unit];
      x.part_len = p.slot_indptr[x.unit + 1] - p.slot_indptr[x.unit];
    } else {
      x.list_base = static_cast<int64_t>(x.unit) * p.topk;
      x.part_len = p.topk;
    }
  } else {
    if (p.qo_indptr != nullptr) {
      x.tok0 = p.qo_indptr[x.unit];
      x.qlen = p.qo_indptr[x.unit + 1] - x.tok0;
    }
    x.part_len = p.seq_lens[x.unit];
  }
  x.rows_total = x.qlen * x.H;
  x.row0 = tile * kRows;
  if (x.row0 >= x.rows_total) return;  // both CTAs take this branch together
  if (p.items != nullptr) {
    x.seg_start = item_begin;
    x.seg_end = min(item_end, x.part_len);
  } else {
    const int span = p.num_segments * p.tile_size;
    const int tps = x.part_len > 0 ? cdiv(x.part_len, span) : 0;
    const int seg_len = tps * p.tile_size;
    x.seg_start = x.seg * seg_len;
    x.seg_end = min(x.seg_start + seg_len, x.part_len);
  }
  x.n_chunks = x.seg_end > x.seg_start ? cdiv(x.seg_end - x.seg_start, kKeys) : 0;

  x.bar0 = smem_u32(smem + kOffBar);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + kOffTslot);
  x.abort = reinterpret_cast<volatile int*>(smem + kOffAbort);
  if (x.tid == 0) {
    *x.abort = 0;
    const uint32_t sharers = SPARSE ? 1 : 2;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(x.bar(kFull + s), 1);
      mbar_init(x.bar(kEmpty + s), sharers);
    }
    for (int s = 0; s < kRSlots; ++s) {
      mbar_init(x.bar(kRFull + s), 1);
      mbar_init(x.bar(kREmpty + s), sharers);
    }
    mbar_init(x.bar(kQFull), 1);
    mbar_init(x.bar(kQTmem), 2 * kSoftWarps);
    mbar_init(x.bar(kSFull), 1);
    mbar_init(x.bar(kSFree), kSoftWarps);
    mbar_init(x.bar(kPFull), kSoftWarps);
    mbar_init(x.bar(kPFree), 1);
    for (int q = 0; q < 4; ++q) mbar_init(x.bar(kX + q), 2);
    mbar_init(x.bar(kDrain), 1);
    mbar_init(x.bar(kDrainPV), 1);
    fence_barrier_init();
  }
  if (x.tid < kSlots + kRSlots) reinterpret_cast<int*>(smem + kOffIssued)[x.tid] = -1;
  if (x.warp == 1) {
    tmem_alloc(smem_u32(tslot), kTmemCols);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before any remote arrive or load
  fence_after_sync();
  x.tbase = *tslot;

  if (x.warp >= 4 && x.warp < 12) {
    softmax_rows<SPARSE>(x, maps, p);
  } else if (x.warp == 1) {
    qk_issue<SPARSE>(x, maps);
  } else if (x.warp == 3) {
    pv_issue<SPARSE>(x);
  } else {
    const int pidx = x.warp == 0 ? 0 : (x.warp == 2 ? 1 : x.warp - 10);
    if constexpr (SPARSE)
      produce_sparse(x, maps, p, pidx);
    else
      produce_dense(x, maps, p, pidx);
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (x.warp == 1) tmem_dealloc(x.tbase, kTmemCols);
  // every load into this CTA's shared memory must have landed before it
  // exits: per slot, the latest use issued here or by the peer, whose record
  // is read once it has stopped issuing (all were consumed unless a wait gave
  // up); then q
  cluster_sync();
  if (x.tid == 0 && x.n_chunks > 0) {
    const volatile int* issued = reinterpret_cast<const volatile int*>(smem + kOffIssued);
    for (int e = 0; e < kSlots + kRSlots; ++e) {
      int last = issued[e];
      if constexpr (!SPARSE)
        last = max(last, ld_cluster_s32(map_to_rank(smem_u32(smem + kOffIssued + 4 * e), x.rank ^ 1)));
      if (last >= 0) drain_wait(x, x.bar(e < kSlots ? kFull + e : kRFull + e - kSlots), last & 1, 12);
    }
    drain_wait(x, x.bar(kQFull), 0, 13);
  }
  cluster_sync();  // no CTA exits while loads into the other may still land
}

template <bool SPARSE>
cudaError_t launch_variant(const VsMaps& maps, const DecodeParams& p, dim3 grid, int* status, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(decode_vs_kernel<SPARSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  decode_vs_kernel<SPARSE><<<grid, kThreads, kSmem, stream>>>(maps, p, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_vs(const DecodeParams& p, int64_t q_rows, int64_t kv_rows, dim3 grid, int* status,
                             cudaStream_t stream) {
  if (p.kv_scales == nullptr) return cudaErrorInvalidValue;
  const bool sparse = p.slots != nullptr;
  VsMaps maps{};
  cudaError_t e = make_row_map(&maps.q, p.q, static_cast<uint64_t>(q_rows), kRows, true);
  if (e == cudaSuccess) e = make_row_map(&maps.qr, p.q, static_cast<uint64_t>(q_rows), kRows, true, 64);
  if (e == cudaSuccess) e = make_row_map(&maps.kv, p.kv, static_cast<uint64_t>(kv_rows), sparse ? 1 : kHalf, true);
  if (e == cudaSuccess) e = make_row_map(&maps.kvr, p.kv, static_cast<uint64_t>(kv_rows), sparse ? 1 : kHalf, true, 64);
  if (e == cudaSuccess && p.out != nullptr)
    e = make_out_map(&maps.out, p.out, static_cast<uint64_t>(q_rows), 1, true, 64, 32, true);
  if (e == cudaSuccess && p.segm_out != nullptr)
    e = p.items != nullptr
            ? make_out_map(&maps.part, p.segm_out, static_cast<uint64_t>(p.segm_rows), 1, false, 32, 32, true)
            : make_out_map(&maps.part, p.segm_out, static_cast<uint64_t>(q_rows),
                           static_cast<uint64_t>(p.num_segments), false, 32, 32, true);
  if (e != cudaSuccess) return e;
  return sparse ? launch_variant<true>(maps, p, grid, status, stream)
                : launch_variant<false>(maps, p, grid, status, stream);
}

}  // namespace mla

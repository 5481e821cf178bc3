// decode_tc.cu -- split-K paged MLA decode on tcgen05 tensor cores (sm_103a).
//
// A CTA pair (thread-block cluster of 2) owns one (128-row tile, segment,
// request), or, under the balanced schedule, the work item its blockIdx
// selects from the list the schedule kernel wrote (request, tile, key range,
// partial slot). Rows are (token, head) pairs of the request; all of them
// share one pass over each KV page. The pair splits the work by stage, so that the
// only traffic between the two SMs is the probabilities:
//   score CTA (rank 0) -- S_g = Q K_g^T over all 576 columns of a 128-key
//       group (M=128, N=128, fp32 in TMEM, two buffers; kind::f16 with q's
//       512 latent dims resident in TMEM and its rope box in shared memory,
//       or kind::f8f6f4 with all of q resident in TMEM). The keys stream
//       through a ring of 16 KB box slots (one 128-byte column box of a
//       group per slot), each slot released by the commit of its own MMAs.
//       Then the masks and a base-2 online softmax with a lazily moved
//       reference max, per 64-key chunk, and P_c (bf16, f16 for e4m3) plus
//       one rescale factor per row go to the value CTA's shared memory: one
//       4 KB + 128 B bulk copy per softmax warp;
//   value CTA (rank 1) -- O += P_c V_c over the 512 value columns (P from
//       shared memory, V an MN-major operand, N=256 twice), O = 128 x 512
//       fp32 filling its whole TMEM; rows whose reference max moved are
//       rescaled in TMEM before the product; the epilogue scales O by the
//       per-row factor the score CTA sends at the end.
// Warps: 0 TMA (q, block-table lookup, key boxes), 1 MMA issue, 2-5
// softmax (score CTA) or O rescale + epilogue (value CTA), 6-9 sparse row
// gathers (TMA gather4, four 128-byte rows per lane), e4m3 -> f16 widening
// of the value columns (value CTA, e4m3) or more TMA producers (6-8): one
// warp issuing TMA loads moves only ~27 bytes per SM clock, several keep the
// SM's load path busy. The value CTA re-reads
// the first 512 columns of each row, which the score CTA has just pulled
// through L2.
// Every wait is bounded; on a timeout the kernel records an error code in
// the status word, stops issuing work, drains what it issued and exits.
#include <atomic>
#include <cfloat>
#include <climits>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "internal.h"
#include "tc_ops.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace tc;

constexpr int kRows = 128;
constexpr int kKeys = 64;                        // keys per P.V chunk (value CTA)
constexpr int kGroup = 128;                      // keys per QK^T (N of the score MMA)
constexpr int kBoxQ = kRows * 128;               // 128 rows x 128 bytes
constexpr int kBox = kKeys * 128;                // 64 rows x 128 bytes
constexpr int kSlot = kGroup * 128;              // ring slot: one 128-byte box of a key group
constexpr int kPBytes = kRows * 128;             // P tile: 128 rows x 64 keys x 16 bit
constexpr int kMsgBytes = kPBytes + kRows * 4;   // P + one rescale factor per row
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0;     // score CTA: scores, 2 buffers x 128 columns
constexpr uint32_t kTmemQ = 256;   // score CTA: q (bf16: 512 latent dims in 256 columns;
                                   // e4m3: 640 dims, zero past 576, in 160 columns)
constexpr uint32_t kTmemO = 0;     // value CTA: O, 512 columns
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kMaxSlots = 16;

enum : int {
  // addressed by the peer CTA
  kPRecvFree = 0, kPFull = 2, kFinal = 4, kDrain = 5,
  // score CTA
  kSFull = 6, kSFree = 8, kQFull = 10, kQTmem = 11, kRFull = 12, kREmpty = 12 + kMaxSlots,
  kScoreBars = 12 + 2 * kMaxSlots,
  // value CTA
  kVFull = 6, kVEmpty = 9, kOReady = 12, kPvDone = 14, kOFinal = 16, kV16Full = 17, kValueBars = 19
};

// Shared-memory header at the same offsets in both CTAs: a CTA addresses
// its peer's barriers, rescale factors and final multipliers through them.
constexpr int kOffBar = 0;
constexpr int kOffTslot = 384;
constexpr int kOffAbort = 388;
constexpr int kOffMult = 512;    // value CTA: final per-row multiplier (128 fp32)
constexpr int kOffAlpha = 1024;  // 2 slots x 128 fp32 rescale factors (received / staged)
constexpr int kHeader = 2048;
static_assert(kScoreBars * 8 <= kOffTslot && kValueBars * 8 <= kOffTslot, "barrier space");

template <bool FP8, bool SPARSE>
struct Cfg {
  // warps 0 and 6-8 issue TMA loads where 6-9 have no other work
  static constexpr int kThreads = 320;
  static constexpr int kProdK = 4;             // score CTA key-ring producer warps
  static constexpr int kProdV = FP8 ? 1 : 4;   // value CTA stage producer warps
  static constexpr int kBoxCols = FP8 ? 128 : 64;  // elements per 128-byte box row
  static constexpr int kBoxesK = FP8 ? 5 : 9;      // score CTA: 576 columns (+ zero fill)
  static constexpr int kBoxesV = FP8 ? 4 : 8;      // value CTA: 512 columns
  static constexpr int kStagesV = FP8 ? 2 : 3;
  static constexpr int kUsable = 232448 - 1024;    // dynamic shared memory minus alignment slack
  // score CTA: q (bf16: the rope box; e4m3: all 5 boxes), the key ring, P staging
  static constexpr int kOffQ = kHeader;
  static constexpr int kOffRing = kOffQ + (FP8 ? 0 : 1) * kBoxQ;
  static constexpr int kBoxesQTmem = FP8 ? 5 : 8;  // q boxes staged through ring slots into TMEM
  static constexpr int kSlots = (kUsable - kOffRing - 2 * kPBytes) / kSlot;
  static constexpr int kOffPStage = kOffRing + kSlots * kSlot;
  static constexpr int kScoreEnd = kOffPStage + 2 * kPBytes;
  // value CTA
  static constexpr int kOffPRecv = kHeader;
  static constexpr int kOffV = kOffPRecv + 2 * kPBytes;
  static constexpr int kOffV16 = kOffV + kStagesV * kBoxesV * kBox;  // e4m3: 2 x 8 f16 boxes
  static constexpr int kValueEnd = kOffV16 + (FP8 ? 2 * 8 * kBox : 0);
  static constexpr int kSmem = (kScoreEnd > kValueEnd ? kScoreEnd : kValueEnd) + 1024;
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kSlots <= kMaxSlots && kSlots >= kBoxesK, "ring slots");
  static_assert(kSlots >= kBoxesQTmem, "q is staged through the first ring slots");
};

struct TcMaps {
  CUtensorMap q;     // q viewed as [T*H rows, 576], box 128 bytes x 128 rows
  CUtensorMap kv;    // cache viewed as [NB*BS rows, 576], box 128 bytes x 64 rows
  CUtensorMap kv1;   // sparse: the same view, box 128 bytes x 1 row (gather4)
  CUtensorMap out;   // out as [T*H, 1, 512] bf16, box 32 rows x 64 columns, 128-byte swizzle
  CUtensorMap part;  // partials as [slot rows, 1, 512] or [T*H, NS, 512] fp32, box 32 x 32
};

__device__ __forceinline__ void report(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// Everything a role needs about its (tile, segment, unit).
struct Ctx {
  uint8_t* smem;
  uint32_t bar0;        // this CTA's barrier 0
  uint32_t peer;        // shared::cluster address of the peer's shared-memory base
  volatile int* abort;
  int* status;
  uint64_t limit_ns;    // bound on each wait (drains keep kTimeoutNs)
  uint32_t tbase;
  int tid, warp, lane;
  int H, tok0, qlen, row0, rows_total, part_len;
  int64_t list_base;
  int seg, seg_start, seg_end, n_chunks, unit;
  int pslot;  // balanced schedule: partial slot of this piece, -1 = write out/lse
  bool fin;   // write the output (else base-2 partials)
  // keys of the segment before the first one that some row of the tile does not see
  // (its first row sees least) or that does not exist
  __device__ int seen_by_all() const { return min(seg_end, part_len - qlen + row0 / H + 1) - seg_start; }
  __device__ uint32_t bar(int i) const { return bar0 + 8u * i; }
  __device__ uint32_t peer_bar(int i) const { return peer + kOffBar + 8u * i; }
};

// Bounded wait on a local barrier phase; `cluster` selects acquire.cluster
// (barriers the peer CTA arrives on or copies into). False on timeout/abort.
// The thread sleeps in the wait (woken by the phase) instead of spinning: a
// spinning warp takes issue slots from the MMA issuer (measured: the
// DeepSeek-V3 batch's decode 125.6 -> 113.3 us).
__device__ bool wait_phase(const Ctx& x, uint32_t bar, uint32_t parity, bool cluster, int code) {
  if (cluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  const uint32_t nap = x.limit_ns < 20000u ? static_cast<uint32_t>(x.limit_ns) : 20000u;
  for (;;) {
    const bool ok = cluster ? mbar_try_wait_cluster_sleep(bar, parity, nap) : mbar_try_wait_sleep(bar, parity, nap);
    if (ok) return true;
    if (*x.abort) return false;
    if (global_timer_ns() - t0 > x.limit_ns) {
      report(x.status, code);
      *x.abort = 1;
      return false;
    }
  }
}

// Wait that ignores the abort flag (teardown drains), still bounded.
__device__ void drain_wait(int* status, uint32_t bar, uint32_t parity, int code) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
    if (global_timer_ns() - t0 > kTimeoutNs) {
      report(status, code);
      return;
    }
  }
}

template <bool F16>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  if constexpr (F16) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Cache row of key position `pos` (dense: 64 keys from a 64-aligned position
// lie in one block, block_size being a multiple of 64).
__device__ __forceinline__ int cache_row(const DecodeParams& p, const int32_t* bt_row, int pos) {
  const int bs = p.block_size;
  const int blk = pos / bs;
  return bt_row[blk] * bs + (pos - blk * bs);
}

// ------------------------------------------------------------------ score CTA: q
// q's boxes land in the first ring slots (bf16: the 8 latent boxes; e4m3:
// all 5, the last half zero-filled past column 576) and are copied into TMEM
// by the softmax warps, which then free the ring; the bf16 rope box stays in
// shared memory.
template <bool FP8, bool SPARSE>
__device__ void load_q(const Ctx& x, const TcMaps& maps) {
  using C = Cfg<FP8, SPARSE>;
  tma_prefetch_desc(&maps.q);
  const int qrow = x.tok0 * x.H + x.row0;
  mbar_arrive_expect_tx(x.bar(kQFull), (FP8 ? 5 : 9) * kBoxQ);
  if constexpr (FP8) {
    for (int j = 0; j < 5; ++j)
      tma_load_2d(smem_u32(x.smem + C::kOffRing + j * kSlot), &maps.q, 128 * j, qrow, x.bar(kQFull));
  } else {
    for (int j = 0; j < 8; ++j)
      tma_load_2d(smem_u32(x.smem + C::kOffRing + j * kSlot), &maps.q, 64 * j, qrow, x.bar(kQFull));
    tma_load_2d(smem_u32(x.smem + C::kOffQ), &maps.q, 512, qrow, x.bar(kQFull));
  }
}

// ------------------------------------------------------------------ score CTA: key ring (dense)
// Box j of key group g (128 keys, two 64-row TMA boxes from their blocks)
// goes to ring slot i % kSlots, i = g * kBoxesK + j. The boxes are dealt
// round-robin to kProdK producer warps (one issuing warp moves ~27 bytes
// per clock; several keep the SM's load path busy).
template <bool FP8, bool SPARSE>
__device__ void score_ring_tma(const Ctx& x, const TcMaps& maps, const DecodeParams& p, int pidx) {
  using C = Cfg<FP8, SPARSE>;
  const int32_t* bt_row = p.block_table + static_cast<int64_t>(x.unit) * p.bt_stride;
  const int n_groups = cdiv(x.n_chunks, 2);
  tma_prefetch_desc(&maps.kv);
  // bf16: slots 0..7 hold q until the softmax warps have copied it to TMEM
  if (n_groups > 0 && !wait_phase(x, x.bar(kQTmem), 0, false, 10)) return;
  int i = 0;
  bool ok = true;
  for (int g = 0; g < n_groups && ok; ++g) {
    const int pos0 = x.seg_start + g * kGroup;
    const int row0 = cache_row(p, bt_row, pos0);
    const bool two = pos0 + kKeys < x.seg_end;
    const int row1 = two ? cache_row(p, bt_row, pos0 + kKeys) : 0;
    for (int j = 0; j < C::kBoxesK; ++j, ++i) {
      if (i % C::kProdK != pidx) continue;
      const int slot = i % C::kSlots;
      const int use = i / C::kSlots;
      if (use >= 1 && !wait_phase(x, x.bar(kREmpty + slot), (use - 1) & 1, false, 11)) {
        ok = false;
        break;
      }
      const uint32_t dst = smem_u32(x.smem + C::kOffRing + slot * kSlot);
      mbar_arrive_expect_tx(x.bar(kRFull + slot), two ? kSlot : kBox);
      if (j == C::kBoxesK - 1) {  // the rope columns: their only read
        const uint64_t pol = l2_evict_first();
        tma_load_2d_hint(dst, &maps.kv, C::kBoxCols * j, row0, x.bar(kRFull + slot), pol);
        if (two) tma_load_2d_hint(dst + kBox, &maps.kv, C::kBoxCols * j, row1, x.bar(kRFull + slot), pol);
      } else {  // latent columns, read again by the value CTA
        tma_load_2d(dst, &maps.kv, C::kBoxCols * j, row0, x.bar(kRFull + slot));
        if (two) tma_load_2d(dst + kBox, &maps.kv, C::kBoxCols * j, row1, x.bar(kRFull + slot));
      }
    }
  }
  // every load this warp issued must have landed before the CTA exits
  for (int k = max(0, i - C::kSlots); k < i; ++k)
    if (k % C::kProdK == pidx) drain_wait(x.status, x.bar(kRFull + k % C::kSlots), (k / C::kSlots) & 1, 12);
}

// ------------------------------------------------------------------ score CTA: key ring (sparse)
// Four gather warps. Box i = g * kBoxesK + j (128 keys of group g, columns
// 64j..64j+63) goes to ring slot i % kSlots and is fetched by warp i % 4:
// lane l issues one TMA gather4 of rows 4l..4l+3 (four 128-byte row pieces,
// swizzled like a tile box), so one warp instruction moves the whole box.
// Keys with slot -1 or past the segment read cache row 0: their scores are
// masked by the softmax warps whatever the row holds.
template <bool SPARSE>
__device__ void score_ring_gather(const Ctx& x, const TcMaps& maps, const DecodeParams& p, int pidx) {
  using C = Cfg<false, SPARSE>;
  const int lane = x.lane;
  const int n_groups = cdiv(x.n_chunks, 2);
  tma_prefetch_desc(&maps.kv1);
  if (n_groups > 0 &&
      !__all_sync(0xffffffffu, wait_phase(x, x.bar(kQTmem), 0, false, 15)))
    return;
  int i = 0;
  bool ok = true;
  for (int g = 0; g < n_groups && ok; ++g) {
    int r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int pos = x.seg_start + g * kGroup + 4 * lane + k;
      const int slot_id = pos < x.seg_end ? p.slots[x.list_base + pos] : -1;
      r[k] = slot_id >= 0 ? slot_id : 0;
    }
    for (int j = 0; j < C::kBoxesK; ++j, ++i) {
      if (i % C::kProdK != pidx) continue;
      const int slot = i % C::kSlots;
      const int use = i / C::kSlots;
      if (use >= 1) {
        ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kREmpty + slot), (use - 1) & 1, false, 14));
        if (!ok) break;
      }
      if (lane == 0) mbar_arrive_expect_tx(x.bar(kRFull + slot), kSlot);
      __syncwarp();
      const uint32_t dst = smem_u32(x.smem + C::kOffRing + slot * kSlot + 512 * lane);
      if (j == C::kBoxesK - 1)  // the rope columns: their only read
        tma_gather4_hint(dst, &maps.kv1, 64 * j, r[0], r[1], r[2], r[3], x.bar(kRFull + slot), l2_evict_first());
      else
        tma_gather4(dst, &maps.kv1, 64 * j, r[0], r[1], r[2], r[3], x.bar(kRFull + slot));
    }
  }
  // every gather this warp issued must have landed before the CTA exits
  if (lane == 0)
    for (int k = max(0, i - C::kSlots); k < i; ++k)
      if (k % C::kProdK == pidx) drain_wait(x.status, x.bar(kRFull + k % C::kSlots), (k / C::kSlots) & 1, 12);
  __syncwarp();
}

// ------------------------------------------------------------------ value CTA: stages (dense)
// Producer warp pidx loads the boxes j = pidx, pidx + kProdV, ... of every
// stage; the stage's barrier completes with all kProdV arrivals and bytes.
template <bool FP8, bool SPARSE>
__device__ void value_stage_tma(const Ctx& x, const TcMaps& maps, const DecodeParams& p, int pidx) {
  using C = Cfg<FP8, SPARSE>;
  const int32_t* bt_row = p.block_table + static_cast<int64_t>(x.unit) * p.bt_stride;
  const int nbox = (C::kBoxesV - pidx + C::kProdV - 1) / C::kProdV;
  tma_prefetch_desc(&maps.kv);
  int issued = 0;
  for (int c = 0; c < x.n_chunks; ++c) {
    const int st = c % C::kStagesV;
    if (c >= C::kStagesV &&
        !wait_phase(x, x.bar(kVEmpty + st), (c / C::kStagesV - 1) & 1, false, 16))
      break;
    const int row = cache_row(p, bt_row, x.seg_start + c * kKeys);
    mbar_arrive_expect_tx(x.bar(kVFull + st), nbox * kBox);
    // the value columns' last read: first out of L2
    const uint64_t pol = l2_evict_first();
    for (int j = pidx; j < C::kBoxesV; j += C::kProdV)
      tma_load_2d_hint(smem_u32(x.smem + C::kOffV + (st * C::kBoxesV + j) * kBox), &maps.kv,
                       C::kBoxCols * j, row, x.bar(kVFull + st), pol);
    issued = c + 1;
  }
  for (int c = max(0, issued - C::kStagesV); c < issued; ++c)
    drain_wait(x.status, x.bar(kVFull + c % C::kStagesV), (c / C::kStagesV) & 1, 17);
}

// ------------------------------------------------------------------ value CTA: stages (sparse)
// Four gather warps; warp w fetches value boxes w and w + 4 of each 64-key
// chunk: lane l issues one TMA gather4 of rows 4(l % 16)..4(l % 16) + 3 of
// box w + 4 (l / 16). A key with slot -1 or past the segment reads the row of
// the chunk's first valid key (its P is zero, and that row is finite wherever
// the exact result is); a chunk without a valid key is zero-filled by stores.
template <bool SPARSE>
__device__ void value_stage_gather(const Ctx& x, const TcMaps& maps, const DecodeParams& p, int pidx) {
  using C = Cfg<false, SPARSE>;
  static_assert(C::kBoxesV == 2 * C::kProdV, "two value boxes per gather warp");
  const int lane = x.lane;
  const int jbox = pidx + C::kProdV * (lane >> 4);
  tma_prefetch_desc(&maps.kv1);
  int issued = 0;
  for (int c = 0; c < x.n_chunks; ++c) {
    const int st = c % C::kStagesV;
    if (c >= C::kStagesV) {
      const bool ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kVEmpty + st),
                                                         (c / C::kStagesV - 1) & 1, false, 18));
      if (!ok) break;
    }
    int r[4];
    int first = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int pos = x.seg_start + c * kKeys + 4 * (lane & 15) + k;
      r[k] = pos < x.seg_end ? p.slots[x.list_base + pos] : -1;
      if (first < 0 && r[k] >= 0) first = r[k];
    }
    const uint32_t have = __ballot_sync(0xffffffffu, first >= 0) & 0xffffu;
    uint8_t* stage = x.smem + C::kOffV + st * C::kBoxesV * kBox;
    if (have != 0) {
      const int sub = __shfl_sync(0xffffffffu, first, __ffs(have) - 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = r[k] >= 0 ? r[k] : sub;
      if (lane == 0) mbar_arrive_expect_tx(x.bar(kVFull + st), 2 * kBox);
      __syncwarp();
      tma_gather4_hint(smem_u32(stage + jbox * kBox + 512 * (lane & 15)), &maps.kv1, 64 * jbox, r[0], r[1],
                       r[2], r[3], x.bar(kVFull + st), l2_evict_first());  // last read of these rows
    } else {
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      for (int b = 0; b < 2; ++b)
        for (int q = lane; q < kBox / 16; q += 32)
          reinterpret_cast<uint4*>(stage + (pidx + C::kProdV * b) * kBox)[q] = z;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(x.bar(kVFull + st));
    }
    issued = c + 1;
  }
  if (lane == 0)
    for (int c = max(0, issued - C::kStagesV); c < issued; ++c)
      drain_wait(x.status, x.bar(kVFull + c % C::kStagesV), (c / C::kStagesV) & 1, 17);
  __syncwarp();
}

// ------------------------------------------------------------------ score CTA: MMA
// S_g (128 rows x 128 keys) into TMEM buffer g & 1: per key box, 4 MMAs of
// K = 16 (bf16, A = q in TMEM; the rope box with A in shared memory) or 4 of
// K = 32 (e4m3, A in shared memory); each box's slot is released by its own
// commit. Descriptors are a base plus compile-time offsets.
template <bool FP8, bool SPARSE>
__device__ void score_mma(const Ctx& x) {
  using C = Cfg<FP8, SPARSE>;
  if (x.lane != 0) return;
  const uint32_t idesc = FP8 ? instr_desc(kRows, kGroup, 0, 0, false, false)
                             : instr_desc(kRows, kGroup, 1, 1, false, false);
  const uint64_t q_desc = smem_desc_sw128(smem_u32(x.smem + C::kOffQ), 16, 1024);
  const uint64_t ring_desc = smem_desc_sw128(smem_u32(x.smem + C::kOffRing), 16, 1024);
  const int n_groups = cdiv(x.n_chunks, 2);
  bool ok = n_groups == 0 || wait_phase(x, x.bar(kQTmem), 0, false, 21);
  int i = 0;
  for (int g = 0; g < n_groups && ok; ++g) {
    const int b = g & 1;
    if (g >= 2 && !wait_phase(x, x.bar(kSFree + b), ((g - 2) >> 1) & 1, false, 23)) break;
    const uint32_t d = x.tbase + kTmemS + 128 * b;
#pragma unroll
    for (int j = 0; j < C::kBoxesK; ++j, ++i) {
      const int slot = i % C::kSlots;
      if (!wait_phase(x, x.bar(kRFull + slot), (i / C::kSlots) & 1, false, 22)) {
        ok = false;
        break;
      }
      fence_after_sync();
      const uint64_t bd = ring_desc + static_cast<uint64_t>(slot * (kSlot >> 4));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t acc = (j | k) != 0 ? 1u : 0u;
        if constexpr (FP8) {  // A = q in TMEM: 8 columns per 32 e4m3 dims
          mma_ts_f8(d, x.tbase + kTmemQ + 32 * j + 8 * k, bd + 2 * k, idesc, acc);
        } else if (j < 8) {
          mma_ts(d, x.tbase + kTmemQ + 32 * j + 8 * k, bd + 2 * k, idesc, acc);
        } else {
          mma_ss(d, q_desc + 2 * k, bd + 2 * k, idesc, acc);
        }
      }
      mma_commit(x.bar(kREmpty + slot));
    }
    if (!ok) break;
    mma_commit(x.bar(kSFull + b));
  }
  mma_commit(x.bar(kDrain));
  drain_wait(x.status, x.bar(kDrain), 0, 24);
}

// ------------------------------------------------------------------ score CTA: softmax
template <bool FP8, bool SPARSE>
__device__ void score_softmax(const Ctx& x, const DecodeParams& p) {
  using C = Cfg<FP8, SPARSE>;
  const int lane = x.lane;
  const int q4 = x.warp & 3;               // TMEM lane quarter of this warp
  const int r = q4 * 32 + lane;            // row within the tile
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const int H = x.H;
  const int rho = x.row0 + r;
  const bool row_ok = rho < x.rows_total;
  const int vis = !row_ok ? 0 : (SPARSE ? INT_MAX : x.part_len - x.qlen + rho / H + 1);
  const float scale2 = p.score_scale_log2;
  bool ok = true;
  if (x.n_chunks > 0) {
    // this row of q, staged by TMA in the first ring slots, into TMEM
    // (bf16: the 512 latent dims as packed pairs, 8 x 32 columns; e4m3: all
    // 576 dims packed four to a column, 5 x 32 columns); then the ring is free
    ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kQFull), 0, false, 30));
    if (ok) {
#pragma unroll 1
      for (int j = 0; j < C::kBoxesQTmem; ++j) {
        const uint8_t* src = x.smem + C::kOffRing + j * kSlot + r * 128;
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
      mbar_arrive(x.bar(kQTmem));
    }
  }
  uint8_t* pstage = x.smem + C::kOffPStage;
  float* alpha_st = reinterpret_cast<float*>(x.smem + kOffAlpha);
  const uint32_t pstage_u = smem_u32(pstage);
  const uint32_t alpha_u = smem_u32(alpha_st);
  float m_ref = -INFINITY, m_true = -INFINITY, l = 0.f;
  int sent = 0;
  for (int c = 0; c < x.n_chunks && ok; ++c) {
    const int b = c & 1;           // P staging / receive slot
    const int g = c >> 1;          // key group of the chunk and its S buffer g & 1
    ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kSFull + (g & 1)), (g >> 1) & 1, false, 31));
    if (!ok) break;
    fence_after_sync();
    float s[64];
    {
      uint32_t sr[64];
      tmem_ld_32x32b_x64(x.tbase + lane_off + kTmemS + 128 * (g & 1) + 64 * (c & 1), sr);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 64; ++j) s[j] = __uint_as_float(sr[j]);
    }
    if ((c & 1) || c + 1 == x.n_chunks) {  // QK^T of group g + 2 may overwrite the buffer
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(x.bar(kSFree + (g & 1)));
    }
    // keys of the chunk that exist: inside the segment and, for the sparse
    // variant, with a valid slot (one ballot per 32 keys)
    const int c0 = x.seg_start + c * kKeys;
    const int nvalid = min(kKeys, x.seg_end - c0);
    uint64_t kmask = nvalid >= 64 ? ~0ull : ((1ull << nvalid) - 1ull);
    if constexpr (SPARSE) {
      const bool v0 = lane < nvalid && p.slots[x.list_base + c0 + lane] >= 0;
      const bool v1 = lane + 32 < nvalid && p.slots[x.list_base + c0 + 32 + lane] >= 0;
      kmask = static_cast<uint64_t>(__ballot_sync(0xffffffffu, v0)) |
              (static_cast<uint64_t>(__ballot_sync(0xffffffffu, v1)) << 32);
    }
    // mask (only chunks with keys that do not exist or are causally hidden)
    // and the chunk maximum over the raw scores (scale2 > 0), 8-way tree
    const int lim = min(x.seg_end, vis) - c0;
    if (lim < 64 || kmask != ~0ull) {
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (!(j < lim && ((kmask >> j) & 1ull))) s[j] = -INFINITY;
    }
    float m8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m8[i] = s[i];
#pragma unroll
    for (int j = 8; j < 64; ++j) m8[j & 7] = fmaxf(m8[j & 7], s[j]);
    const float mraw = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                             fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
    const float mx = mraw * scale2;  // -inf stays -inf
    m_true = fmaxf(m_true, mx);
    float alpha = 1.f;
    if (mx > m_ref + 8.f) {
      if (m_ref != -INFINITY) {
        alpha = fast_exp2(m_ref - mx);
        l *= alpha;
      }
      m_ref = mx;
    }
    // P = 2^(s * scale2 - m_ref); 8 partial sums
    const float base = m_ref == -INFINITY ? 0.f : m_ref;
    uint32_t pk[32];
    float ps8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) ps8[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float p0 = fast_exp2(fmaf(s[2 * j], scale2, -base));
      const float p1 = fast_exp2(fmaf(s[2 * j + 1], scale2, -base));
      ps8[j & 7] += p0 + p1;
      pk[j] = pack_p<FP8>(p0, p1);
    }
    l += ((ps8[0] + ps8[1]) + (ps8[2] + ps8[3])) + ((ps8[4] + ps8[5]) + (ps8[6] + ps8[7]));
    // P row and rescale factor into staging buffer b (K-major, 128-byte
    // swizzle), once the copy of chunk c - 2 has read it
    if (lane == 0) bulk_wait_read<1>();
    __syncwarp();
    uint8_t* prow = pstage + b * kPBytes + r * 128;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      *reinterpret_cast<uint4*>(prow + ((q ^ (r & 7)) << 4)) =
          make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
    alpha_st[b * kRows + r] = alpha;
    fence_proxy_async_smem();
    __syncwarp();
    bool okc = true;
    if (lane == 0) {
      // the value CTA's slot b is free once its P.V of chunk c - 2 completed
      if (c >= 2) okc = wait_phase(x, x.bar(kPRecvFree + b), ((c - 2) >> 1) & 1, true, 32);
      if (okc) {
        const uint32_t full = x.peer_bar(kPFull + b);
        bulk_copy_to_cluster(x.peer + C::kOffPRecv + b * kPBytes + q4 * 4096,
                             pstage_u + b * kPBytes + q4 * 4096, 4096, full);
        bulk_copy_to_cluster(x.peer + kOffAlpha + (b * kRows + q4 * 32) * 4,
                             alpha_u + (b * kRows + q4 * 32) * 4, 128, full);
        bulk_commit_group();
      }
    }
    ok = __shfl_sync(0xffffffffu, okc ? 1 : 0, 0) != 0;
    if (ok) sent = c + 1;
  }

  // ------------------------------------------------------------ final factors
  if (ok) {
    const int tok = x.tok0 + (row_ok ? rho / H : 0);
    const int head = row_ok ? rho % H : 0;
    const int64_t th = static_cast<int64_t>(tok) * H + head;
    float mult;
    float lse = -INFINITY;
    if (x.fin) {
      if (p.sinks != nullptr) {
        const float s2 = p.sinks[head] * kLog2e;
        const float M = fmaxf(m_ref, s2);
        const float e = l > 0.f ? exp2f(m_ref - M) : 0.f;
        const float W = l * e + (s2 == -INFINITY ? 0.f : exp2f(s2 - M));  // (-inf: no sink; NaN stays)
        mult = W != 0.f ? e / W : 0.f;
        if (W != 0.f) lse = kLn2 * (M + log2f(W));
      } else if (l != 0.f) {  // (a NaN stays)
        mult = 1.f / l;
        lse = kLn2 * (m_ref + log2f(l));
      } else {
        mult = 0.f;
      }
    } else {
      mult = l != 0.f ? 1.f / l : 0.f;
    }
    if (row_ok) {
      if (x.fin) {
        p.lse[th] = lse;
      } else {
        const int64_t ts = x.pslot >= 0 ? static_cast<int64_t>(x.pslot) * p.slot_rows + r
                                        : th * p.num_segments + x.seg;
        const float2 part = partial_sums(l > 0.f ? m_true : -INFINITY, l > 0.f ? l * exp2f(m_ref - m_true) : l);
        p.segm_max[ts] = part.x;
        p.segm_expsum[ts] = part.y;
      }
    }
    st_cluster_f32(x.peer + kOffMult + 4 * r, mult * p.kv_scale);
    mbar_arrive_cluster(x.peer_bar(kFinal));
  }
  // Teardown: the value CTA's commits for the last chunks arrive on this
  // CTA's barriers, and the copies must have left this CTA's staging.
  if (lane == 0) {
    if (x.warp == 2) {
      for (int c = max(0, sent - 2); c < sent; ++c)
        drain_wait(x.status, x.bar(kPRecvFree + (c & 1)), (c >> 1) & 1, 37);
    }
    bulk_wait_all();
  }
}

// ------------------------------------------------------------------ value CTA: MMA
template <bool FP8, bool SPARSE>
__device__ void value_mma(const Ctx& x) {
  using C = Cfg<FP8, SPARSE>;
  if (x.lane != 0) return;
  const uint32_t idesc = FP8 ? instr_desc(kRows, 256, 0, 0, false, true)
                             : instr_desc(kRows, 256, 1, 1, false, true);
  const uint64_t p_desc = smem_desc_sw128(smem_u32(x.smem + C::kOffPRecv), 16, 1024);
  const uint64_t v_desc = smem_desc_sw128(smem_u32(x.smem + (FP8 ? C::kOffV16 : C::kOffV)), kBox, 1024);
  const int n = x.n_chunks;
  bool ok = true;
  for (int c = 0; c < n && ok; ++c) {
    const int st = c % C::kStagesV;
    const int slot = c & 1;
    const uint32_t par = (c >> 1) & 1;
    ok = FP8 ? wait_phase(x, x.bar(kV16Full + slot), par, false, 41)
             : wait_phase(x, x.bar(kVFull + st), (c / C::kStagesV) & 1, false, 41);
    ok = ok && wait_phase(x, x.bar(kPFull + slot), par, true, 42);
    if (!ok) break;
    // re-arm the slot for chunk c + 2 (its phase completes with the copies)
    if (c + 2 < n) mbar_arrive_expect_tx(x.bar(kPFull + slot), kMsgBytes);
    if (!wait_phase(x, x.bar(kOReady + slot), par, false, 43)) break;
    fence_after_sync();
    const uint64_t vb = v_desc + static_cast<uint64_t>((FP8 ? slot * 8 : st * 8) * (kBox >> 4));
    const uint64_t pb = p_desc + static_cast<uint64_t>(slot * (kPBytes >> 4));
#pragma unroll
    for (int ks = 0; ks < kKeys / 16; ++ks) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        mma_ss(x.tbase + kTmemO + 256 * h, pb + 2 * ks,
               vb + static_cast<uint64_t>((h * 4 * kBox + ks * 2048) >> 4), idesc,
               (c | ks) != 0 ? 1u : 0u);
    }
    if (!FP8) mma_commit(x.bar(kVEmpty + st));
    mma_commit_mc(x.bar(kPRecvFree + slot), 0x1);  // the score CTA may refill the slot
    mma_commit(x.bar(kPvDone + slot));
  }
  if (ok && n >= 1) mma_commit(x.bar(kOFinal));
  mma_commit(x.bar(kDrain));
  drain_wait(x.status, x.bar(kDrain), 0, 44);
}

// ------------------------------------------------------------------ value CTA: rescale + epilogue
template <bool FP8, bool SPARSE>
__device__ void value_rows(const Ctx& x, const TcMaps& maps, const DecodeParams& p) {
  using C = Cfg<FP8, SPARSE>;
  const int lane = x.lane;
  const int q4 = x.warp & 3;
  const int r = q4 * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const int H = x.H;
  const float* alpha_rx = reinterpret_cast<const float*>(x.smem + kOffAlpha);
  const int n = x.n_chunks, seen = x.seen_by_all();
  bool ok = true;
  for (int c = 0; c < n && ok; ++c) {
    const int slot = c & 1;
    ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kPFull + slot), (c >> 1) & 1, true, 51));
    if (!ok) break;
    const float a = alpha_rx[slot * kRows + r];
    if (__any_sync(0xffffffffu, a != 1.f)) {
      // this warp's O rows are relative to an old reference: wait for
      // P.V of chunk c - 1, then rescale them in TMEM
      if (c >= 1) {
        ok = __all_sync(0xffffffffu,
                        wait_phase(x, x.bar(kPvDone + ((c - 1) & 1)), ((c - 1) >> 1) & 1, false, 52));
        if (!ok) break;
      }
      fence_after_sync();
#pragma unroll 1
      for (int g = 0; g < 8; ++g) {
        uint32_t o[64];
        tmem_ld_32x32b_x64(x.tbase + lane_off + kTmemO + 64 * g, o);
        tmem_ld_wait();
        uint32_t o0[32], o1[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          o0[j] = __float_as_uint(__uint_as_float(o[j]) * a);
          o1[j] = __float_as_uint(__uint_as_float(o[32 + j]) * a);
        }
        tmem_st_32x32b_x32(x.tbase + lane_off + kTmemO + 64 * g, o0);
        tmem_st_32x32b_x32(x.tbase + lane_off + kTmemO + 64 * g + 32, o1);
      }
      tmem_st_wait();
    }
    if constexpr (!FP8 && !SPARSE) {
      // The segment's last chunk may end inside the page: zero the value
      // rows past the segment so that whatever the cache holds there cannot
      // reach O through P = 0; nor may what is not finite in the values of keys
      // that only later tokens see.
      const int from = seen - c * kKeys;
      if (from < kKeys) {
        const int nvalid = x.seg_end - (x.seg_start + c * kKeys);
        const int st = c % C::kStagesV;
        ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kVFull + st), (c / C::kStagesV) & 1, false, 53));
        if (!ok) break;
        uint8_t* vst = x.smem + C::kOffV + st * C::kBoxesV * kBox;
        static_assert(C::kBoxesV == 8, "64 pieces of 16 bytes a row");
        for (int i = max(from, 0) * 64 + x.tid - 64; i < kKeys * 64; i += 128) {
          const int row = i >> 6;
          uint4* at = reinterpret_cast<uint4*>(vst + ((i >> 3) & 7) * kBox + row * 128 + (i & 7) * 16);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (row < nvalid) {
            v = *at;
            v = make_uint4(bf16x2_finite(v.x), bf16x2_finite(v.y), bf16x2_finite(v.z), bf16x2_finite(v.w));
          }
          *at = v;
        }
        fence_proxy_async_smem();
      }
    }
    fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kOReady + slot));
  }

  // ------------------------------------------------------------ epilogue
  if (ok && n > 0) {
    ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kOFinal), 0, false, 54));
    fence_after_sync();
  }
  if (ok) ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kFinal), 0, true, 55));
  // Each warp scales its 32 rows and stages them, 128 bytes of each row at a
  // time, in its quarter of a P slot (no P arrives after the last chunk), in
  // the 128-byte swizzle. When all 32 rows are valid one TMA tensor store
  // writes each staged tile (two tiles in flight, one per P slot), so that
  // the warp never waits on global stores. Otherwise every store
  // instruction covers four 128-byte row pieces. TMEM loads are
  // warp-collective (ok is warp-uniform).
  if (ok) {
    const float mult = reinterpret_cast<const float*>(x.smem + kOffMult)[r];
    uint8_t* stg = x.smem + C::kOffPRecv + ((n - 1) & 1) * kPBytes + q4 * 4096;
    const bool whole = x.row0 + 32 * q4 + 32 <= x.rows_total && n > 0;
    if (whole) {
      // the warp's rows are consecutive rows of out, of the item's partial
      // slot, or of the segment's partials
      const int wr = x.row0 + 32 * q4;
      const int z0 = x.fin || x.pslot < 0 ? x.tok0 * H + wr : x.pslot * p.slot_rows + 32 * q4;
      const int y0 = x.fin || x.pslot >= 0 ? 0 : x.seg;
      const CUtensorMap* map = x.fin ? &maps.out : &maps.part;
      int staged = 0;
      auto store = [&](const uint32_t (&w)[32], int col0) {
        uint8_t* buf = x.smem + C::kOffPRecv + ((n - 1 + staged) & 1) * kPBytes + q4 * 4096;
        if (staged >= 2) {  // the store that read this tile two passes ago
          if (lane == 0) bulk_wait_read<1>();
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<uint4*>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) =
              make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(map, smem_u32(buf), col0, y0, z0);
          bulk_commit_group();
        }
        ++staged;
      };
#pragma unroll 1
      for (int g = 0; g < 8; ++g) {
        uint32_t o[64];
        tmem_ld_32x32b_x64(x.tbase + lane_off + kTmemO + 64 * g, o);
        tmem_ld_wait();
        if (x.fin) {
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 32; ++j)
            w[j] = pack_bf16(__uint_as_float(o[2 * j]) * mult, __uint_as_float(o[2 * j + 1]) * mult);
          store(w, 64 * g);
        } else {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(o[32 * hf + j]) * mult);
            store(w, 64 * g + 32 * hf);
          }
        }
      }
      if (lane == 0) bulk_wait_all();  // tiles read and written before the CTA exits
      __syncwarp();
      return;
    }
    const int qc = lane & 7;  // 16-byte piece of a 128-byte row piece
    // output bases (16-byte units) of the 8 rows this lane writes, rows
    // 4 * it + lane / 8 of the warp's 32; null past the last valid row
    uint4* rbase[8];
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int rr = x.row0 + 32 * q4 + 4 * it + (lane >> 3);
      rbase[it] = nullptr;
      if (rr < x.rows_total) {
        const int64_t th = static_cast<int64_t>(x.tok0 + rr / H) * H + rr % H;
        const int64_t ts = x.pslot >= 0 ? static_cast<int64_t>(x.pslot) * p.slot_rows + (rr - x.row0)
                                        : th * p.num_segments + x.seg;
        rbase[it] = x.fin ? reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + th * kRank)
                          : reinterpret_cast<uint4*>(p.segm_out + ts * kRank);
      }
    }
    // one 32-row x 128-byte tile: this lane's row in, four rows per store out
    auto pass = [&](const uint32_t (&w)[32], int unit0) {
      __syncwarp();  // the previous pass has read the staging tile
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4*>(stg + lane * 128 + ((q ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
      __syncwarp();
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int row = 4 * it + (lane >> 3);
        const uint4 v = *reinterpret_cast<const uint4*>(stg + row * 128 + ((qc ^ (row & 7)) << 4));
        if (rbase[it] != nullptr) rbase[it][unit0 + qc] = v;
      }
    };
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {
      // 16-byte units of column group g: 8 per bf16 row piece, 16 per fp32
      const int gu = x.fin ? 8 * g : 16 * g;
      if (n == 0) {  // no key: zeros, written straight out (coalesced)
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          if (rbase[it] == nullptr) continue;
          rbase[it][gu + qc] = z;
          if (!x.fin) rbase[it][gu + 8 + qc] = z;
        }
        continue;
      }
      uint32_t o[64];
      tmem_ld_32x32b_x64(x.tbase + lane_off + kTmemO + 64 * g, o);
      tmem_ld_wait();
      if (x.fin) {
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
          w[j] = pack_bf16(__uint_as_float(o[2 * j]) * mult, __uint_as_float(o[2 * j + 1]) * mult);
        pass(w, gu);
      } else {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(o[32 * hf + j]) * mult);
          pass(w, gu + 8 * hf);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ value CTA: e4m3 widening
// 128 threads widen the chunk's 512 e4m3 value columns (4 boxes) to f16 (8
// boxes, exact) in buffer c & 1, zeroing rows past the segment, and NaNs of
// keys that only later tokens see.
template <bool SPARSE>
__device__ void widen_values(const Ctx& x) {
  using C = Cfg<true, SPARSE>;
  const int ct = x.tid - 192, seen = x.seen_by_all();
  bool ok = true;
  for (int c = 0; c < x.n_chunks && ok; ++c) {
    const int st = c % C::kStagesV;
    const int slot = c & 1;
    ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kVFull + st), (c / C::kStagesV) & 1, false, 61));
    if (!ok) break;
    if (c >= 2) {  // P.V of chunk c - 2 has finished reading buffer slot
      ok = __all_sync(0xffffffffu, wait_phase(x, x.bar(kPvDone + slot), ((c - 2) >> 1) & 1, false, 62));
      if (!ok) break;
    }
    const int nvalid = min(kKeys, x.seg_end - (x.seg_start + c * kKeys));
    const int from = seen - c * kKeys;
    const uint8_t* src = x.smem + C::kOffV + st * C::kBoxesV * kBox;
    uint8_t* dst = x.smem + C::kOffV16 + slot * 8 * kBox;
    for (int i = ct; i < C::kBoxesV * kKeys * 8; i += 128) {
      const int box = i >> 9;
      const int rem = i & 511;
      const int row = rem >> 3;
      const int k = rem & 7;  // logical 16-byte chunk (16 e4m3 values)
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (row < nvalid)
        v = *reinterpret_cast<const uint4*>(src + box * kBox + row * 128 + ((k ^ (row & 7)) << 4));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t hh[8];
#pragma unroll
      for (int e2 = 0; e2 < 4; ++e2) {
        hh[2 * e2] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[e2] & 0xFFFF));
        hh[2 * e2 + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[e2] >> 16));
      }
      if (row >= from) {
#pragma unroll
        for (int e = 0; e < 8; ++e) hh[e] = f16x2_without_nan(hh[e]);
      }
      const int lc = (k & 3) * 2;
      uint8_t* drow = dst + (box * 2 + (k >> 2)) * kBox + row * 128;
      *reinterpret_cast<uint4*>(drow + ((lc ^ (row & 7)) << 4)) = make_uint4(hh[0], hh[1], hh[2], hh[3]);
      *reinterpret_cast<uint4*>(drow + (((lc + 1) ^ (row & 7)) << 4)) = make_uint4(hh[4], hh[5], hh[6], hh[7]);
    }
    fence_proxy_async_smem();
    mbar_arrive(x.bar(kVEmpty + st));
    mbar_arrive(x.bar(kV16Full + slot));
  }
}

template <bool FP8, bool SPARSE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<FP8, SPARSE>::kThreads, 1)
    decode_tc_kernel(const __grid_constant__ TcMaps maps, const DecodeParams p, int* status) {
  using C = Cfg<FP8, SPARSE>;
  static_assert(!(FP8 && SPARSE), "the sparse variant is bf16");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctx x;
  x.smem = smem;
  x.status = status;
  x.limit_ns = p.wait_ns != 0 ? p.wait_ns : kTimeoutNs;
  x.tid = threadIdx.x;
  x.warp = x.tid >> 5;
  x.lane = x.tid & 31;
  const uint32_t crank = cluster_ctarank();
  const bool score = crank == 0;
  int tile, item_begin = 0, item_end = 0;
  x.pslot = -1;
  if (p.items != nullptr) {
    // balanced schedule: both CTAs of the pair read the same item, once the
    // grid that wrote the list has completed (a no-op unless this grid was
    // launched as a programmatic dependent of it)
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    // the merge grid may launch once every CTA of this one has started (it
    // waits for this grid to complete before it reads)
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
  x.part_len = 0;
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
    if (p.shared != 0) {  // tokens and visible keys of the item itself (of a prefix: all keys for all rows)
      const int4 b = reinterpret_cast<const int4*>(p.items)[2 * (blockIdx.x >> 1) + 1];
      x.tok0 = b.y;
      x.qlen = b.z & kItemTokens;
      x.part_len = (b.z & kItemPrefix) != 0 ? INT_MAX : b.w + x.qlen - 1;
    }
  }
  x.rows_total = x.qlen * x.H;
  x.row0 = tile * kRows;
  if (x.row0 >= x.rows_total) return;  // both CTAs of the pair take this branch together

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
    if (score) {
      for (int s = 0; s < C::kSlots; ++s) {
        mbar_init(x.bar(kRFull + s), 1);
        mbar_init(x.bar(kREmpty + s), 1);
      }
      for (int b = 0; b < 2; ++b) {
        mbar_init(x.bar(kSFull + b), 1);
        mbar_init(x.bar(kSFree + b), 4);
        mbar_init(x.bar(kPRecvFree + b), 1);
      }
      mbar_init(x.bar(kQFull), 1);
      mbar_init(x.bar(kQTmem), 128);
    } else {
      for (int s = 0; s < C::kStagesV; ++s) {
        mbar_init(x.bar(kVFull + s), C::kProdV);
        // e4m3: free once widened (128 arrivals); else the P.V commit
        mbar_init(x.bar(kVEmpty + s), FP8 ? 128 : 1);
      }
      for (int b = 0; b < 2; ++b) {
        mbar_init(x.bar(kPFull + b), 1);
        mbar_init(x.bar(kOReady + b), 4);
        mbar_init(x.bar(kPvDone + b), 1);
        mbar_init(x.bar(kV16Full + b), 128);
      }
      mbar_init(x.bar(kOFinal), 1);
      mbar_init(x.bar(kFinal), 128);
    }
    mbar_init(x.bar(kDrain), 1);
    fence_barrier_init();
    // the first two receive slots expect the score CTA's copies
    if (!score)
      for (int b = 0; b < 2 && b < x.n_chunks; ++b) mbar_arrive_expect_tx(x.bar(kPFull + b), kMsgBytes);
  }
  if (x.warp == 1) {
    tmem_alloc(smem_u32(tslot), kTmemCols);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before any remote arrive or copy
  fence_after_sync();
  x.tbase = *tslot;
  x.peer = map_to_rank(smem_u32(smem), crank ^ 1u);

  // producer index of warps 0, 6, 7, 8 (-1: not a producer)
  const int pidx = x.warp == 0 ? 0 : (x.warp >= 6 && x.warp <= 8 ? x.warp - 5 : -1);
  if (score) {
    if (x.warp == 0) {
      if (x.lane == 0 && x.n_chunks > 0) {
        load_q<FP8, SPARSE>(x, maps);
        if (!SPARSE) score_ring_tma<FP8, SPARSE>(x, maps, p, 0);
        drain_wait(status, x.bar(kQFull), 0, 13);
      }
    } else if (x.warp == 1) {
      score_mma<FP8, SPARSE>(x);
    } else if (x.warp < 6) {
      score_softmax<FP8, SPARSE>(x, p);
    } else if constexpr (SPARSE) {
      if (x.warp >= 6 && x.n_chunks > 0) score_ring_gather<SPARSE>(x, maps, p, x.warp - 6);
    } else {
      if (pidx >= 1 && pidx < C::kProdK && x.lane == 0 && x.n_chunks > 0)
        score_ring_tma<FP8, SPARSE>(x, maps, p, pidx);
    }
  } else {
    if (x.warp == 1) {
      value_mma<FP8, SPARSE>(x);
    } else if (x.warp >= 2 && x.warp < 6) {
      value_rows<FP8, SPARSE>(x, maps, p);
    } else if constexpr (SPARSE) {
      if (x.warp >= 6) value_stage_gather<SPARSE>(x, maps, p, x.warp - 6);
    } else if constexpr (FP8) {
      if (x.warp == 0 && x.lane == 0) value_stage_tma<FP8, SPARSE>(x, maps, p, 0);
      if (x.warp >= 6) widen_values<SPARSE>(x);
    } else {
      if (pidx >= 0 && pidx < C::kProdV && x.lane == 0) value_stage_tma<FP8, SPARSE>(x, maps, p, pidx);
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // no remote access to this CTA's shared memory after here
  fence_after_sync();
  if (x.warp == 1) tmem_dealloc(x.tbase, kTmemCols);
}

template <bool FP8, bool SPARSE>
cudaError_t launch_variant(const TcMaps& maps, const DecodeParams& p, dim3 grid, int* status,
                           cudaStream_t stream) {
  using C = Cfg<FP8, SPARSE>;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(decode_tc_kernel<FP8, SPARSE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  // an ordinary launch also after the schedule kernel: as a programmatic
  // dependent of it (set up while it runs) the DeepSeek-V3 call measured
  // 137.8 us against 131.0 us (its griddepcontrol.wait is then a no-op)
  decode_tc_kernel<FP8, SPARSE><<<grid, C::kThreads, C::kSmem, stream>>>(maps, p, status);
  return cudaGetLastError();
}

}  // namespace

int decode_tc_smem_bytes(bool fp8) {
  return fp8 ? Cfg<true, false>::kSmem : Cfg<false, false>::kSmem;
}

cudaError_t launch_decode_tc(const DecodeParams& p, bool fp8, int64_t q_rows, int64_t kv_rows,
                             dim3 grid, int* status, cudaStream_t stream) {
  TcMaps maps{};
  cudaError_t e = make_row_map(&maps.q, p.q, static_cast<uint64_t>(q_rows), kRows, fp8);
  if (e != cudaSuccess) return e;
  e = make_row_map(&maps.kv, p.kv, static_cast<uint64_t>(kv_rows), kKeys, fp8);
  if (e != cudaSuccess) return e;
  if (p.out != nullptr) {
    e = make_out_map(&maps.out, p.out, static_cast<uint64_t>(q_rows), 1, true, 64, 32, true);
    if (e != cudaSuccess) return e;
  }
  if (p.segm_out != nullptr) {
    e = p.items != nullptr
            ? make_out_map(&maps.part, p.segm_out, static_cast<uint64_t>(p.segm_rows), 1, false, 32, 32, true)
            : make_out_map(&maps.part, p.segm_out, static_cast<uint64_t>(q_rows),
                           static_cast<uint64_t>(p.num_segments), false, 32, 32, true);
    if (e != cudaSuccess) return e;
  }
  if (p.slots != nullptr) {
    if (fp8) return cudaErrorNotSupported;
    e = make_row_map(&maps.kv1, p.kv, static_cast<uint64_t>(kv_rows), 1, false);
    if (e != cudaSuccess) return e;
    return launch_variant<false, true>(maps, p, grid, status, stream);
  }
  return fp8 ? launch_variant<true, false>(maps, p, grid, status, stream)
             : launch_variant<false, false>(maps, p, grid, status, stream);
}

}  // namespace mla

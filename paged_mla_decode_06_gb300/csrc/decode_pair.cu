// decode_pair.cu -- attention of a batch that shares prefixes, over an e4m3 cache
// (with or without group scales), for tiles of 128 query rows: two CTAs that
// share every matrix instruction of a tile (sm_103a, cta_group::2).
//
// All query rows that see the same keys make one matrix: the rows of a group's
// tokens over its prefix, and those of a request over its own keys. An item of the work list is a
// tile of 128 of them and a range of keys. The fp32 accumulator of 128 rows x
// 512 value columns fills a whole tensor memory, so a tile takes two SMs. Here
// the pair splits the rows: M = 128 over two CTAs gives each 64 rows and, in
// either half of its TMEM lanes, half of an instruction's columns, so that 64
// rows x 512 columns take 256 TMEM columns. Nothing is computed twice, the
// softmax of a row stays in one CTA, and each CTA holds half of every B operand:
// per chunk of 128 keys, with rank r of the pair,
//   S[rows, keys]  = Q K^T   M = 128, N = 128, K = 576: CTA r has its 64 rows of
//                            q, and keys 64 r .. 64 r + 63: 18 kind::f8f6f4
//                            instructions of 46 cycles (measured; of 32 at N = 256,
//                            for whose keys the shared memory has no room);
//   O[rows, 512]  += P V     for j = 0, 1: M = 128, N = 256, K = 128: CTA r has its
//                            rows of P as two terms (hi e5m2, lo e4m3), and value
//                            columns 256 j + 128 r .. + 127 of all 128 keys, read MN-major: 16
//                            instructions of 64.3 cycles.
// That is 1860 tensor cycles a chunk and pair. (The value-split kernel takes 2180,
// having both SMs compute all scores, and 3100 to 3400 in all, bound by its
// softmax of all 128 rows in either SM.) An instruction reads the same
// shared-memory offsets in both CTAs, so a CTA's own keys as B of Q K^T and its
// columns as B of P V cannot share a copy: K and V have rings of their own, and
// a chunk brings 52 KB of keys and values, 16 KB of them twice, into each SM.
//
// The softmax works on chunks: one group of eight warps takes the even ones,
// another the odd ones. TMEM lanes 0..63 hold the rows' scores of keys 0..63,
// lanes 64..127 those of keys 64..127; a warp takes 32 rows x 32 keys, and four
// warps exchange a row's maximum. With t = score + log2 s (KeyScale), the weights
// are p = 2^(t - ref + 4), in two terms: hi in e5m2, the upper byte of p's f16
// rounded there (so that it needs no conversion, and the rest p - hi is exact in
// f16), and the rest in e4m3. That is 7 bits of p down to 2^-3, 3 bits down to
// 2^-14. The rest fits e4m3 while p < 2^11.8, so the reference moves only when
// a maximum exceeds it by more than 7.75: O is then rescaled in TMEM, which P V
// has to wait for. (hi in e4m3, as the value-split kernel has it, leaves 4.75, and most
// chunks had a row that moved.)
//
// Rank 0 issues all matrix instructions; their completion is committed to the
// barriers of both CTAs. Rank 1's copies complete on its own barriers, and two
// of its warps pass that on to rank 0 (so that either CTA can drain what it
// loaded without the other). Softmax warps arrive on rank 0's barriers, from
// either CTA.
//
// Warps: 0 loads, 1 issues Q K^T (rank 1: passes keys on), 2 prepares the keys'
// scales, 3 issues P V (passes values on), 4-19 softmax and epilogue. Every wait
// is bounded: a timeout records a code in the status word, stops the CTA's
// work, drains what was issued and exits.
#include <atomic>
#include <climits>

#include "common.cuh"
#include "internal.h"
#include "tc_ops.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace tc;

constexpr int kRows = 128;                // query rows of a tile: M
constexpr int kOwnRows = 64;              // of a CTA
constexpr int kKeys = 128;                // keys per chunk
constexpr int kHalf = 64;                 // keys of a CTA as B of Q K^T; K of a step of P V
constexpr int kBox = kHalf * 128;         // 128-byte columns of 64 rows
constexpr int kRBox = kHalf * 64;         // the rope columns of 64 rows
constexpr int kKSlot = 4 * kBox + kRBox;  // a CTA's keys of a chunk
constexpr int kVSlot = 2 * kBox;          // its value columns of an instruction, of all keys
constexpr int kKRing = 2;                 // chunks
constexpr int kVRing = 4;                 // slots: column box j of chunk c is number 2 c + j
constexpr int kSoftWarps = 16;
constexpr int kGroupWarps = 8;
constexpr int kPart = 32;                 // keys of a softmax warp
constexpr int kUni = 16;                  // keys that share their scale where the groups are multiples of it
constexpr int kThreads = 32 * (4 + kSoftWarps);
constexpr int kPTile = kOwnRows * kKeys;  // one term of P of a chunk
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;            // 256 columns: 128 for each j
constexpr uint32_t kTmemS = 256;          // [2] 64: S of chunk c at c % 2
constexpr uint64_t kDefaultWaitNs = 2000000000ull;
constexpr uint32_t kSleepNs = 20000;
constexpr float kPBias = 4.f;
constexpr float kMove = 7.75f;

enum : int {
  kKFull = 0,                  // [kKRing] this CTA's keys of a chunk have landed
  kKEmpty = kKFull + kKRing,   // [kKRing] released by Q K^T
  kVFull = kKEmpty + kKRing,   // [kVRing] a column box of this CTA's values has landed
  kVEmpty = kVFull + kVRing,   // [kVRing] P V over it complete: released, O_j holds the chunk
  kPeerK = kVEmpty + kVRing,   // [kKRing] rank 0: rank 1's keys have landed
  kPeerV = kPeerK + kKRing,    // [kVRing] rank 0: rank 1's values
  kQFull = kPeerV + kVRing,    // this CTA's rows of q
  // of chunk c, at c % 2:
  kSFull,                      // [2] S written and key scales ready
  kSFree = kSFull + 2,         // [2] rank 0: S read by both CTAs
  kPFull = kSFree + 2,         // [2] rank 0: P written by both CTAs, O_0 rescaled
  kOReady = kPFull + 2,        // [2] rank 0: O_1 rescaled
  kX = kOReady + 2,            // [4][2] (at c % 4) the four warps of 32 rows have posted their maxima
  kScFree = kX + 8,            // [2] key scales read
  kXL = kScFree + 2,           // [2] the eight warps of 32 rows have posted their sums
  kDrainQK = kXL + 2,          // Q K^T and P V complete, in both CTAs
  kDrainPV,
  kNumBars
};

// Shared memory.
constexpr int kOffBar = 0;
constexpr int kOffTslot = 448;
constexpr int kOffAbort = 452;
constexpr int kOffIssued = 456;                  // {last chunk of keys, last box of values} issued
constexpr int kOffMask = 480;                    // [2][4] bits of existing keys of chunk c (at c % 2)
constexpr int kOffXMax = 512;                    // [4][4][64] maxima of chunk c (at c % 4) by key quarter
constexpr int kOffScale = kOffXMax + 4096;       // [2][mul, add, inv][128]
constexpr int kOffLsum = kOffScale + 3 * 1024;   // [2][4][64] row sums by group and key quarter
constexpr int kOffQ = 10240;                     // 4 boxes of 64 rows, 128-byte swizzle; rope box, 64-byte swizzle
constexpr int kOffP = kOffQ + kKSlot;            // [c % 2][hi, lo] 64 rows x 128 keys, 128-byte swizzle
constexpr int kOffK = kOffP + 4 * kPTile;
constexpr int kOffV = kOffK + kKRing * kKSlot;
constexpr int kSmem = kOffV + kVRing * kVSlot + 1024;  // + alignment slack
static_assert(kNumBars * 8 <= kOffTslot && kOffLsum + 2048 <= kOffQ, "header space");
static_assert(kSmem <= 232448, "shared memory budget");
static_assert(kKRing * kKSlot + kVRing * kVSlot >= kSoftWarps * 8192, "the epilogue stages in the rings");

struct PairMaps {
  CUtensorMap q;     // q as [T*H rows, 576], box 128 bytes x 64 rows
  CUtensorMap qr;    // the same, box 64 bytes
  CUtensorMap kv;    // cache as [NB*BS rows, 576], box 128 bytes x BOX rows
  CUtensorMap kvr;   // the same, box 64 bytes
  CUtensorMap out;   // out as [T*H, 1, 512] bf16, box 32 rows x 64 columns, 128-byte swizzle
  CUtensorMap part;  // partials as [slot rows, 1, 512] fp32, box 32 x 32
};

// How a key's scale reaches its score: one for the whole cache, one for each 16
// keys in a row (groups of a multiple of 16 slots), one for each key.
enum class Scale { kNone, kSixteen, kKey };

struct Ctx {
  uint8_t* smem;
  uint32_t bar0, lead0;  // barriers of this CTA and of rank 0 (cluster addresses)
  volatile int* abort;
  int* status;
  uint64_t limit_ns;
  uint32_t tbase;
  int tid, warp, lane, rank;
  int H, unit, tok0, row0, rows_total;
  int see0;              // keys that the first token of the unit sees; INT_MAX: all rows see all keys
  int seg_start, seg_end, n_chunks;
  int pslot;             // first row of the partial's slot, -1: write out/lse
  __device__ uint32_t bar(int i) const { return bar0 + 8u * i; }
  __device__ uint32_t lead(int i) const { return lead0 + 8u * i; }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Four weights (in order from the low byte) as two words of codes, the first
// in e5m2, the rest in e4m3. (p is positive and below 2^12: the carry of the
// rounding stays in its half. A NaN goes on in the rest.)
__device__ __forceinline__ void split4(float p0, float p1, float p2, float p3, uint32_t& hi, uint32_t& lo) {
  asm("{\n .reg .b16 l0, l1;\n .reg .b32 a, b, c, d;\n"
      " cvt.rn.f16x2.f32 a, %3, %2;\n cvt.rn.f16x2.f32 b, %5, %4;\n"
      " add.u32 c, a, 0x00800080;\n add.u32 d, b, 0x00800080;\n"
      " and.b32 c, c, 0xff00ff00;\n and.b32 d, d, 0xff00ff00;\n"
      " prmt.b32 %0, c, d, 0x7531;\n"
      " sub.f16x2 a, a, c;\n sub.f16x2 b, b, d;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l0, a;\n cvt.rn.satfinite.e4m3x2.f16x2 l1, b;\n"
      " mov.b32 %1, {l0, l1};\n}\n"
      : "=r"(hi), "=r"(lo)
      : "f"(p0), "f"(p1), "f"(p2), "f"(p3));
}

// ------------------------------------------------------------------ pair instructions
__device__ __forceinline__ void pair_alloc(uint32_t dst_saddr, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst_saddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive once on the barrier at this offset in both CTAs when every MMA this
// thread issued so far has completed.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// ------------------------------------------------------------------ waits
__device__ __forceinline__ void report(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// Bounded wait on a barrier phase, sleeping; false on timeout (recorded) or
// abort. Barriers that the other CTA arrives on are waited for as the CTA's own:
// no thread reads what one of the other CTA wrote through the generic proxy (P,
// S and O are read by the tensor core of the SM that holds them, after proxy and
// tcgen05 fences), and acquire and release at cluster scope took 1000 to 2000 cycles
// each (168 us against 192 for 64 requests over 8192 common keys, 128 heads).
__device__ bool wait_phase(const Ctx& x, uint32_t bar, uint32_t parity, int code) {
  const bool brief = x.limit_ns < kSleepNs;  // (a sleep may last longer than the limit: poll)
  if (mbar_test_wait(bar, parity)) return true;
  if (!brief && mbar_try_wait_sleep(bar, parity, kSleepNs)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!(brief ? mbar_test_wait(bar, parity) : mbar_try_wait_sleep(bar, parity, kSleepNs))) {
    if (*x.abort) return false;
    if (global_timer_ns() - t0 > x.limit_ns) {
      report(x.status, code);
      *x.abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool warp_wait(const Ctx& x, uint32_t bar, uint32_t parity, int code) {
  return __all_sync(0xffffffffu, wait_phase(x, bar, parity, code)) != 0;
}
// Wait that ignores the abort flag (teardown), still bounded.
__device__ void drain_wait(const Ctx& x, uint32_t bar, uint32_t parity, int code) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_sleep(bar, parity, kSleepNs)) {
    if (global_timer_ns() - t0 > kDefaultWaitNs) {
      report(x.status, code);
      return;
    }
  }
}

// ------------------------------------------------------------------ keys
// Cache rows of the runs of BOX keys that share a TMA box: looked up by the
// whole warp, 32 runs at a time and a window ahead. A run past the end or in a
// column without a block has row -BOX: a box that is filled with zeros.
template <int BOX>
struct RowWindow {
  static constexpr int kPer = kKeys / BOX;   // runs of a chunk
  static constexpr int kSpan = 32 / kPer;    // chunks of a window
  int cur, nxt;
  __device__ __forceinline__ int look(const Ctx& x, const DecodeParams& p, const int32_t* bt_row, int w0) const {
    const int pos = x.seg_start + w0 * kKeys + x.lane * BOX;
    if (pos >= x.seg_end) return -BOX;
    const int blk = pos / p.block_size;
    const int b = bt_row[blk];
    return b < 0 ? -BOX : b * p.block_size + (pos - blk * p.block_size);
  }
  __device__ __forceinline__ void start(const Ctx& x, const DecodeParams& p, const int32_t* bt_row) {
    cur = look(x, p, bt_row, 0);
    nxt = look(x, p, bt_row, kSpan);
  }
  // moves on to the window of chunk c (called for every chunk in turn)
  __device__ __forceinline__ void at(const Ctx& x, const DecodeParams& p, const int32_t* bt_row, int c) {
    if (c > 0 && c % kSpan == 0) {
      cur = nxt;
      nxt = look(x, p, bt_row, c + kSpan);
    }
  }
  __device__ __forceinline__ int row(int c, int run) const {
    return __shfl_sync(0xffffffffu, cur, kPer * (c % kSpan) + run);
  }
};

// Warp 0: the keys of each chunk (five column boxes of this CTA's 64 rows) and its
// values (two column boxes of all 128 rows), each as soon as
// its slot is free; the boxes of a kind go out together, one lane each. (In
// turn, the keys of a chunk waited behind the values of the one before, whose
// slots P V frees late: 4600 cycles a chunk. A warp more for either would leave 80
// registers a thread.)
template <int BOX>
__device__ void load_boxes(const Ctx& x, const PairMaps& maps, const DecodeParams& p) {
  constexpr int kSub = kHalf / BOX;  // boxes high of 64 rows
  const int box = x.lane / kSub, run = x.lane % kSub;
  const int32_t* bt_row = p.block_table + static_cast<int64_t>(x.unit) * p.bt_stride;
  volatile int* issued = reinterpret_cast<volatile int*>(x.smem + kOffIssued);
  const uint32_t base = smem_u32(x.smem);
  RowWindow<BOX> kw, vw;
  kw.start(x, p, bt_row);
  vw = kw;
  uint64_t t0 = 0;
  int polls = 0;
  for (int c = 0, g = 0; g < 2 * x.n_chunks;) {
    bool idle = true;
    if (c < x.n_chunks) {
      const int s = c % kKRing;
      if (c < kKRing || __all_sync(0xffffffffu, mbar_test_wait(x.bar(kKEmpty + s), (c / kKRing - 1) & 1))) {
        kw.at(x, p, bt_row, c);
        if (x.lane == 0) {
          mbar_arrive_expect_tx(x.bar(kKFull + s), kKSlot);
          issued[0] = c;
        }
        __syncwarp();
        const int row = kw.row(c, x.rank * kSub + run);
        const uint32_t to = base + kOffK + s * kKSlot;
        if (box < 4) tma_load_2d(to + box * kBox + run * BOX * 128, &maps.kv, 128 * box, row, x.bar(kKFull + s));
        if (box == 4) tma_load_2d(to + 4 * kBox + run * BOX * 64, &maps.kvr, kRank, row, x.bar(kKFull + s));
        __syncwarp();
        ++c;
        idle = false;
      }
    }
    {
      const int s = g % kVRing;
      if (g < kVRing || __all_sync(0xffffffffu, mbar_test_wait(x.bar(kVEmpty + s), (g / kVRing - 1) & 1))) {
        if ((g & 1) == 0) vw.at(x, p, bt_row, g >> 1);
        if (x.lane == 0) {
          mbar_arrive_expect_tx(x.bar(kVFull + s), kVSlot);
          issued[1] = g;
        }
        __syncwarp();
        const int vrun = x.lane % (2 * kSub);  // (of 128 rows)
        const int row = vw.row(g >> 1, vrun);
        if (x.lane < 2 * kSub)
          tma_load_2d(base + kOffV + s * kVSlot + vrun * BOX * 128, &maps.kv, 128 * (2 * (g & 1) + x.rank), row,
                      x.bar(kVFull + s));
        __syncwarp();
        ++g;
        idle = false;
      }
    }
    if (!idle) {
      t0 = 0;
      polls = 0;
      continue;
    }
    __nanosleep(40);
    if ((++polls & 63) != 0) continue;  // (reading the global timer takes longer than most waits)
    const uint64_t now = __shfl_sync(0xffffffffu, global_timer_ns(), 0);
    if (t0 == 0) t0 = now;
    if (__shfl_sync(0xffffffffu, *x.abort, 0)) break;
    if (now - t0 > x.limit_ns) {
      if (x.lane == 0) {
        report(x.status, 11);
        *x.abort = 1;
      }
      break;
    }
  }
  __syncwarp();
}

__device__ __forceinline__ float scale_of_slot(const DecodeParams& p, int s) {
  const uint32_t g = p.scale_magic != 0 ? __umulhi(static_cast<uint32_t>(s), p.scale_magic) >> p.scale_shift
                                        : static_cast<uint32_t>(s) >> p.scale_shift;
  return __ldg(p.kv_scales + g);
}

// Warp 2: the scales of a chunk's keys and the bits of those that exist, read one
// chunk ahead of the one posted, each once the softmax has read those two chunks back.
template <int BOX, Scale SCALE>
__device__ void prepare_keys(const Ctx& x, const DecodeParams& p) {
  const int lane = x.lane;
  const int32_t* bt_row = p.block_table + static_cast<int64_t>(x.unit) * p.bt_stride;
  RowWindow<BOX> w;
  w.start(x, p, bt_row);
  float sc[4];
  uint32_t bits[4];
  auto read = [&](int c) {
    w.at(x, p, bt_row, c);
    const int n = x.seg_end - (x.seg_start + c * kKeys);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 32 * i + lane;
      const int row = w.row(c, j / BOX);
      const bool there = j < n && row >= 0;
      bits[i] = __ballot_sync(0xffffffffu, there);
      if constexpr (SCALE == Scale::kKey) sc[i] = there ? scale_of_slot(p, row + j % BOX) : 1.f;
    }
    if constexpr (SCALE == Scale::kSixteen) {
      const int j = kUni * (lane & 7);
      const int row = w.row(c, j / BOX);
      sc[0] = j < n && row >= 0 ? scale_of_slot(p, row + j % BOX) : 1.f;
    }
  };
  if (x.n_chunks > 0) read(0);
  for (int c = 0; c < x.n_chunks; ++c) {
    const int b = c & 1;
    if (c >= 2 && !warp_wait(x, x.bar(kScFree + b), ((c >> 1) - 1) & 1, 27)) break;
    float* ks = reinterpret_cast<float*>(x.smem + kOffScale) + b * 3 * kKeys;
    if (lane < 4)
      reinterpret_cast<uint32_t*>(x.smem + kOffMask)[b * 4 + lane] =
          lane == 0 ? bits[0] : lane == 1 ? bits[1] : lane == 2 ? bits[2] : bits[3];
    if constexpr (SCALE != Scale::kNone) {
#pragma unroll
      for (int i = 0; i < (SCALE == Scale::kKey ? 4 : 1); ++i) {
        const KeyScale k = key_scale(sc[i], p.score_scale_log2);
        const int at = SCALE == Scale::kKey ? 32 * i + lane : kUni * lane;
        if (SCALE == Scale::kKey || lane < kKeys / kUni) {
          ks[at] = k.mul;
          ks[kKeys + at] = k.add;
          ks[2 * kKeys + at] = k.inv;
        }
      }
    }
    __syncwarp();
    if (c >= 2 && !warp_wait(x, x.bar(kSFull + b), ((c >> 1) - 1) & 1, 28)) break;  // S two chunks back
    if (lane == 0) mbar_arrive(x.bar(kSFull + b));
    if (c + 1 < x.n_chunks) read(c + 1);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ MMA issue
// Rank 0, warp 1.
__device__ void qk_issue(const Ctx& x) {
  constexpr uint32_t kId = instr_desc(kRows, kKeys, 0, 0, false, false);
  const uint32_t base = smem_u32(x.smem);
  const uint64_t q_desc = smem_desc_sw128(base + kOffQ, 16, 1024);
  const uint64_t qr_desc = smem_desc_sw64(base + kOffQ + 4 * kBox, 512);
  const uint64_t k_desc = smem_desc_sw128(base + kOffK, 16, 1024);
  const uint64_t kr_desc = smem_desc_sw64(base + kOffK + 4 * kBox, 512);
  const bool one = elect_one();
  bool ok = warp_wait(x, x.bar(kQFull), 0, 20);
  for (int c = 0; c < x.n_chunks; ++c) {
    const int b = c & 1, s = c % kKRing;
    ok = ok && warp_wait(x, x.bar(kKFull + s), (c / kKRing) & 1, 23) &&
         warp_wait(x, x.bar(kPeerK + s), (c / kKRing) & 1, 21);
    ok = ok && (c < 2 || warp_wait(x, x.bar(kSFree + b), ((c >> 1) - 1) & 1, 22));
    if (!ok) break;
    fence_after_sync();
    const uint64_t kd = k_desc + static_cast<uint64_t>((s * kKSlot) >> 4);
    const uint64_t krd = kr_desc + static_cast<uint64_t>((s * kKSlot) >> 4);
    const uint32_t d = x.tbase + kTmemS + 64u * b;
    if (one) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint64_t off = static_cast<uint64_t>(((i >> 2) * kBox + (i & 3) * 32) >> 4);
        pair_mma(d, q_desc + off, kd + off, kId, i != 0 ? 1u : 0u);
      }
      pair_mma(d, qr_desc, krd, kId, 1u);
      pair_mma(d, qr_desc + 2, krd + 2, kId, 1u);
      pair_commit(x.bar(kSFull + b));
      pair_commit(x.bar(kKEmpty + s));
    }
    __syncwarp();
  }
  if (one) {
    pair_commit(x.bar(kDrainQK));
    drain_wait(x, x.bar(kDrainQK), 0, 25);
  }
  __syncwarp();
}

// Rank 0, warp 3: P V of a chunk by halves of the columns, so that a half of O may
// be rescaled while the other is multiplied.
__device__ void pv_issue(const Ctx& x) {
  constexpr uint32_t kIdHi = instr_desc(kRows, 256, 1, 0, false, true);
  constexpr uint32_t kIdLo = instr_desc(kRows, 256, 0, 0, false, true);
  const uint32_t base = smem_u32(x.smem);
  const uint64_t v_desc = smem_desc_sw128(base + kOffV, kBox, 1024);  // MN-major
  const uint64_t p_desc = smem_desc_sw128(base + kOffP, 16, 1024);
  const bool one = elect_one();
  bool ok = true;
  for (int g = 0; g < 2 * x.n_chunks && ok; ++g) {
    const int j = g & 1, c = g >> 1, b = c & 1, s = g % kVRing;
    ok = warp_wait(x, x.bar((j == 0 ? kPFull : kOReady) + b), (c >> 1) & 1, j == 0 ? 24 : 38) &&
         warp_wait(x, x.bar(kVFull + s), (g / kVRing) & 1, 26) &&
         warp_wait(x, x.bar(kPeerV + s), (g / kVRing) & 1, 39);
    if (!ok) break;
    fence_after_sync();
    const uint64_t vb = v_desc + static_cast<uint64_t>((s * kVSlot) >> 4);
    const uint64_t pb = p_desc + static_cast<uint64_t>((b * 2 * kPTile) >> 4);
    const uint32_t d = x.tbase + kTmemO + 128u * j;
    if (one) {
#pragma unroll
      for (int ks = 0; ks < kKeys / 32; ++ks) {
        const uint64_t av = pb + static_cast<uint64_t>((ks * 32) >> 4);
        const uint64_t bv = vb + static_cast<uint64_t>((ks * 32 * 128) >> 4);
        pair_mma(d, av, bv, kIdHi, (c | ks) != 0 ? 1u : 0u);
        pair_mma(d, av + static_cast<uint64_t>(kPTile >> 4), bv, kIdLo, 1u);
      }
      pair_commit(x.bar(kVEmpty + s));
    }
    __syncwarp();
  }
  if (one) {
    pair_commit(x.bar(kDrainPV));
    drain_wait(x, x.bar(kDrainPV), 0, 29);
  }
  __syncwarp();
}

// Rank 1, warps 1 and 3: what has landed here, passed on to rank 0.
__device__ void pass_keys(const Ctx& x) {
  bool ok = warp_wait(x, x.bar(kQFull), 0, 20);
  for (int c = 0; c < x.n_chunks && ok; ++c) {
    const int s = c % kKRing;
    ok = warp_wait(x, x.bar(kKFull + s), (c / kKRing) & 1, 23);
    if (ok && x.lane == 0) mbar_arrive_remote(x.lead(kPeerK + s));
    __syncwarp();
  }
  if (x.lane == 0) drain_wait(x, x.bar(kDrainQK), 0, 25);
  __syncwarp();
}
__device__ void pass_values(const Ctx& x) {
  bool ok = true;
  for (int g = 0; g < 2 * x.n_chunks && ok; ++g) {
    const int s = g % kVRing;
    ok = warp_wait(x, x.bar(kVFull + s), (g / kVRing) & 1, 26);
    if (ok && x.lane == 0) mbar_arrive_remote(x.lead(kPeerV + s));
    __syncwarp();
  }
  if (x.lane == 0) drain_wait(x, x.bar(kDrainPV), 0, 29);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax + epilogue
template <Scale SCALE>
__device__ void softmax_rows(const Ctx& x, const PairMaps& maps, const DecodeParams& p) {
  constexpr bool UNI = SCALE == Scale::kSixteen, ONE = SCALE == Scale::kNone;
  const int lane = x.lane;
  const int sw = x.warp - 4;
  const int q4 = x.warp & 3;               // TMEM lane quarter of this warp
  const int rq = q4 & 1;                   // its 32 of the CTA's 64 rows
  const int kq = q4 >> 1;                  // its half of a chunk's keys
  const int h = sw >> 3;                   // chunks c with c % 2 == h, and buffer
  const int kh = (sw >> 2) & 1;            // its 32 keys of the half
  const int part = 2 * kq + kh;            // key quarter (and, of a rescaling, columns of O_kh)
  const int cq = sw >> 2;                  // quarter of the TMEM columns of O at the end
  const int r = rq * 32 + lane;            // row within the CTA
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const int H = x.H;
  const int rho = x.row0 + kOwnRows * x.rank + r;  // row within the unit
  const bool row_ok = rho < x.rows_total;
  const int vis = !row_ok ? 0 : (x.see0 == INT_MAX ? INT_MAX : x.see0 + rho / H);
  // keys from here on (of the segment) are not seen by all rows
  const int all_see = x.see0 == INT_MAX ? INT_MAX : x.see0 + x.row0 / H - x.seg_start;
  const int n = x.n_chunks;
  bool ok = true;

  float* xmax = reinterpret_cast<float*>(x.smem + kOffXMax) + r;
  uint8_t* prow = x.smem + kOffP + h * 2 * kPTile + r * 128;
  const int c0 = ((2 * part) ^ (r & 7)) << 4, c1 = ((2 * part + 1) ^ (r & 7)) << 4;
  const uint32_t ts = x.tbase + lane_off + kTmemS + 64u * h + kPart * kh;

  float ref = -INFINITY, l = 0.f;
  auto follow = [&](float mx) {
    if (!(mx > ref + kMove)) return 1.f;  // (moves also when a row's first visible key arrives)
    const float a = ref == -INFINITY ? 1.f : fast_exp2(ref - mx);
    ref = mx;
    l *= a;
    return a;
  };
  auto row_max = [&](int c) {
    const float* xm = xmax + (c & 3) * 4 * kOwnRows;
    return fmaxf(fmaxf(xm[0], xm[kOwnRows]), fmaxf(xm[2 * kOwnRows], xm[3 * kOwnRows]));
  };
  // the maximum of chunk c, which the other group posted. A group looks at it
  // before it posts its own of c + 1, which the other waits for before it posts
  // that of c + 4: neither the barrier's phase nor the four buffers are passed over.
  auto follow_other = [&](int c) {
    if (!warp_wait(x, x.bar(kX + 2 * (c & 3) + rq), (c >> 2) & 1, 33)) return false;
    follow(row_max(c));
    return true;
  };
  for (int c = h; c < n && ok; c += 2) {
    const int ph = (c >> 1) & 1;
    ok = warp_wait(x, x.bar(kSFull + h), ph, 31);
    if (!ok) break;
    fence_after_sync();
    float s[kPart];
    {
      uint32_t sr[kPart];
      tmem_ld_32x32b_x32(ts, sr);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < kPart; ++j) s[j] = __uint_as_float(sr[j]);
    }
    fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive_remote(x.lead(kSFree + h));  // Q K^T two chunks on may overwrite it
    const float* ks = reinterpret_cast<const float*>(x.smem + kOffScale) + h * 3 * kKeys + kPart * part;
    const uint32_t kmask = reinterpret_cast<const uint32_t*>(x.smem + kOffMask)[4 * h + part];
    if constexpr (SCALE == Scale::kKey) {
#pragma unroll
      for (int j = 0; j < kPart; j += 4) {
        const float4 mu = *reinterpret_cast<const float4*>(ks + j);
        const float4 ad = *reinterpret_cast<const float4*>(ks + kKeys + j);
        const float2 a = fma2(make_float2(s[j], s[j + 1]), make_float2(mu.x, mu.y), make_float2(ad.x, ad.y));
        const float2 b = fma2(make_float2(s[j + 2], s[j + 3]), make_float2(mu.z, mu.w), make_float2(ad.z, ad.w));
        s[j] = a.x;
        s[j + 1] = a.y;
        s[j + 2] = b.x;
        s[j + 3] = b.y;
      }
    }
    // keys that exist and that the row may see
    const int lim = min(vis, x.seg_end) - (x.seg_start + c * kKeys + kPart * part);
    if (lim < kPart || kmask != 0xffffffffu) {
#pragma unroll
      for (int j = 0; j < kPart; ++j)
        if (!(j < lim && ((kmask >> j) & 1u))) s[j] = -INFINITY;
    }
    float m[2];  // of either half of the keys
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* e = s + kUni * i;
      m[i] = fmaxf(max3(max3(e[0], e[1], e[2]), max3(e[3], e[4], e[5]), max3(e[6], e[7], e[8])),
                   max3(max3(e[9], e[10], e[11]), max3(e[12], e[13], e[14]), e[15]));
      if constexpr (UNI) m[i] = fmaf(m[i], ks[kUni * i], ks[kKeys + kUni * i]);  // (mul > 0; -inf stays)
      if constexpr (ONE) m[i] *= p.score_scale_log2;
    }
    // the row's maximum over all key quarters; the previous chunk's before it
    ok = c == 0 || follow_other(c - 1);
    if (!ok) break;
    xmax[((c & 3) * 4 + part) * kOwnRows] = fmaxf(m[0], m[1]);
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kX + 2 * (c & 3) + rq));
    ok = warp_wait(x, x.bar(kX + 2 * (c & 3) + rq), (c >> 2) & 1, 32);
    if (!ok) break;
    const float alpha = follow(row_max(c));
    // p as hi + lo terms, 16 keys to a 16-byte chunk of each tile
    const float base = ref == -INFINITY ? 0.f : ref - kPBias;
    float psum = 0.f;
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mu = UNI ? ks[kUni * i] : ONE ? p.score_scale_log2 : 1.f;
      const float sh = UNI ? ks[kKeys + kUni * i] - base : -base;
      const float2 mul2 = make_float2(mu, mu), shift2 = make_float2(sh, sh);
      float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int j = 4 * i; j < 4 * i + 4; ++j) {
        const int e = 4 * j;
        float2 a = make_float2(s[e], s[e + 1]), b = make_float2(s[e + 2], s[e + 3]);
        a = UNI || ONE ? fma2(a, mul2, shift2) : add2(a, shift2);
        b = UNI || ONE ? fma2(b, mul2, shift2) : add2(b, shift2);
        a = make_float2(fast_exp2(a.x), fast_exp2(a.y));
        b = make_float2(fast_exp2(b.x), fast_exp2(b.y));
        if constexpr (UNI || ONE) {
          ps[0] = add2(ps[0], a);
          ps[1] = add2(ps[1], b);
        } else {
          const float4 iv = *reinterpret_cast<const float4*>(ks + 2 * kKeys + e);
          ps[0] = fma2(a, make_float2(iv.x, iv.y), ps[0]);
          ps[1] = fma2(b, make_float2(iv.z, iv.w), ps[1]);
        }
        split4(a.x, a.y, b.x, b.y, hi[j], lo[j]);
      }
      const float sum = (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y);
      psum = UNI ? fmaf(sum, ks[2 * kKeys + kUni * i], psum) : psum + sum;
    }
    l += psum;
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kScFree + h));
    // P V two chunks back has read this buffer of P
    auto pv_done = [&](int cc, int j, int code) {
      const int g = 2 * cc + j;
      return warp_wait(x, x.bar(kVEmpty + g % kVRing), (g / kVRing) & 1, code);
    };
    ok = c < 2 || pv_done(c - 2, 1, 37);
    if (!ok) break;
    *reinterpret_cast<uint4*>(prow + c0) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(prow + c1) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
    *reinterpret_cast<uint4*>(prow + kPTile + c0) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(prow + kPTile + c1) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
    // Value rows of keys that do not exist (cache rows past the sequence) are
    // zeroed, and of keys that some rows of the tile do not see the NaNs: neither
    // may reach O through p = 0. Each warp sees to the 32 keys of its quarter, a
    // half of them by each of its two row halves.
    if (kmask != 0xffffffffu || all_see < c * kKeys + kPart * (part + 1)) {
#pragma unroll 1
      for (int j = 0; j < 2 && ok; ++j) {
        const int g = 2 * c + j;
        ok = warp_wait(x, x.bar(kVFull + g % kVRing), (g / kVRing) & 1, 36);  // (its writes are seen here too)
        uint8_t* box = x.smem + kOffV + g % kVRing * kVSlot + kPart * part * 128 + (lane & 7) * 16;
        for (int i = rq + 2 * (lane >> 3); ok && i < kPart; i += 8) {
          uint4* at = reinterpret_cast<uint4*>(box + i * 128);
          if (!((kmask >> i) & 1u)) {
            *at = make_uint4(0u, 0u, 0u, 0u);
          } else if (c * kKeys + kPart * part + i >= all_see) {
            const uint4 v = *at;
            *at = make_uint4(e4m3x4_without_nan(v.x), e4m3x4_without_nan(v.y), e4m3x4_without_nan(v.z),
                             e4m3x4_without_nan(v.w));
          }
        }
      }
      if (!ok) break;
    }
    fence_proxy_async_smem();
    const bool moved = __any_sync(0xffffffffu, alpha != 1.f);
    if (kh == 1 && lane == 0) mbar_arrive_remote(x.lead(kPFull + h));  // (P alone)
    if (moved) {
      // some rows moved their reference: once P V of the previous chunk into O_kh
      // is complete, this warp rescales its lanes' rows there
      ok = pv_done(c - 1, kh, 40);
      if (!ok) break;
      fence_after_sync();
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const uint32_t ta = x.tbase + lane_off + kTmemO + 128 * kh + 64 * k;
        uint32_t o[32], o2[32];
        tmem_ld_32x32b_x32(ta, o);
        tmem_ld_32x32b_x32(ta + 32, o2);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          o2[i] = __float_as_uint(__uint_as_float(o2[i]) * alpha);
        }
        tmem_st_32x32b_x32(ta, o);
        tmem_st_32x32b_x32(ta + 32, o2);
      }
      tmem_st_wait();
    }
    fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive_remote(x.lead((kh == 0 ? kPFull : kOReady) + h));
  }

  // ---------------------------------------------------------------- epilogue
  if (ok && n > 0 && ((n - 1) & 1) != h) ok = follow_other(n - 1);  // the last one was the other group's
  float* lsum = reinterpret_cast<float*>(x.smem + kOffLsum) + r;
  if (ok) {
    lsum[(4 * h + part) * kOwnRows] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kXL + rq));
    ok = warp_wait(x, x.bar(kXL + rq), 0, 34);
  }
  // O is complete with the last chunk
  if (ok && n > 0) {
    const int g = 2 * n - 1;
    ok = warp_wait(x, x.bar(kVEmpty + g % kVRing), (g / kVRing) & 1, 35);
    fence_after_sync();
  }
  if (!ok) return;
  const bool fin = x.pslot < 0;
  float mult = 0.f;
  if (row_ok) {
    float L = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) L += lsum[k * kOwnRows];
    const float base = ref == -INFINITY ? 0.f : ref - kPBias;  // the reference of O and the sum
    const int head = rho % H;
    const int64_t th = static_cast<int64_t>(x.tok0 + rho / H) * H + head;
    const bool writes = kq == 0 && cq == 0;
    if (fin) {
      float lse = -INFINITY;
      if (p.sinks != nullptr) {
        const float s2 = p.sinks[head] * kLog2e;
        const float M = fmaxf(L > 0.f ? base : -INFINITY, s2);
        const float e = L > 0.f ? exp2f(base - M) : 0.f;
        const float W = L * e + (s2 == -INFINITY ? 0.f : exp2f(s2 - M));  // (-inf: no sink; NaN stays)
        if (W != 0.f) {
          mult = e / W;
          lse = kLn2 * (M + log2f(W));
        }
      } else if (L != 0.f) {
        mult = 1.f / L;
        lse = kLn2 * (base + log2f(L));
      }
      if (writes) p.lse[th] = lse;
    } else {
      mult = L != 0.f ? 1.f / L : 0.f;
      if (writes) {
        const int64_t at = static_cast<int64_t>(x.pslot) + kOwnRows * x.rank + r;
        const float2 ms = partial_sums(L > 0.f ? base : -INFINITY, L);
        p.segm_max[at] = ms.x;
        p.segm_expsum[at] = ms.y;
      }
    }
    mult *= p.kv_scale;
  }
  // Each warp scales its 32 rows x 64 columns and stages them, 128 bytes of
  // each row at a time, in the 128-byte swizzle, in the rings (which hold no
  // more boxes in use). When all 32 rows are valid one TMA tensor store writes
  // each staged tile; otherwise every store instruction covers four 128-byte row
  // pieces. (TMEM loads are warp-collective.)
  const int col0 = 256 * (cq >> 1) + 128 * kq + 64 * (cq & 1);
  const int wr = x.row0 + kOwnRows * x.rank + 32 * rq;  // the warp's first row within the unit
  if (wr >= x.rows_total) return;
  const bool whole = wr + 32 <= x.rows_total;
  const int z0 = fin ? x.tok0 * H + wr : x.pslot + (wr - x.row0);
  const CUtensorMap* map = fin ? &maps.out : &maps.part;
  const int qc = lane & 7;                  // 16-byte piece of a 128-byte row piece
  auto store = [&](const uint32_t (&w)[32], int col, int tile) {
    uint8_t* buf = x.smem + kOffK + sw * 8192 + tile * 4096;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      *reinterpret_cast<uint4*>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    if (whole) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(map, smem_u32(buf), col, 0, z0);
        bulk_commit_group();
      }
    } else {
      __syncwarp();
#pragma unroll 1
      for (int it = 0; it < 8; ++it) {
        const int row = 4 * it + (lane >> 3);
        if (wr + row >= x.rows_total) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(buf + row * 128 + ((qc ^ (row & 7)) << 4));
        const int64_t at = static_cast<int64_t>(z0 + row) * kRank + col;
        uint8_t* dst = fin ? static_cast<uint8_t*>(p.out) + at * 2 : reinterpret_cast<uint8_t*>(p.segm_out + at);
        *reinterpret_cast<uint4*>(dst + qc * 16) = v;
      }
    }
  };
  auto load = [&](int c, uint32_t (&o)[32]) {
    if (n > 0) {
      tmem_ld_32x32b_x32(x.tbase + lane_off + kTmemO + 64 * cq + 32 * c, o);
      tmem_ld_wait();
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = 0u;
    }
  };
  if (fin) {
    uint32_t w[32];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t o[32];
      load(c, o);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * mult, __uint_as_float(o[2 * j + 1]) * mult);
        w[16 * c + j] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    store(w, col0, 0);
  } else {
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      uint32_t o[32];
      load(c, o);
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * mult);
      store(o, col0 + 32 * c, c);
    }
  }
  if (lane == 0) bulk_wait_read<0>();  // the tiles are read before the CTA exits
  __syncwarp();
}

template <int BOX, Scale SCALE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    decode_pair_kernel(const __grid_constant__ PairMaps maps, const DecodeParams p, int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // the list, once the grid that wrote it has completed; the merge may launch
  // once every CTA has started
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int item = blockIdx.x >> 1;
  if (item >= *p.n_items) return;
  const int4 a = reinterpret_cast<const int4*>(p.items)[2 * item];
  const int4 b = reinterpret_cast<const int4*>(p.items)[2 * item + 1];
  Ctx x;
  x.smem = smem;
  x.status = status;
  x.limit_ns = p.wait_ns != 0 ? p.wait_ns : kDefaultWaitNs;
  x.tid = threadIdx.x;
  x.warp = __shfl_sync(0xffffffffu, x.tid >> 5, 0);  // uniform, for the compiler too
  x.lane = x.tid & 31;
  x.rank = static_cast<int>(cluster_ctarank());
  x.H = p.num_heads;
  x.unit = a.x;
  x.row0 = a.y * kRows;
  x.seg_start = a.z;
  x.seg_end = a.w;
  x.pslot = b.x;
  x.tok0 = b.y;
  x.rows_total = (b.z & kItemTokens) * x.H;
  x.see0 = (b.z & kItemPrefix) != 0 ? INT_MAX : b.w;
  x.n_chunks = x.seg_end > x.seg_start ? cdiv(x.seg_end - x.seg_start, kKeys) : 0;

  x.bar0 = smem_u32(smem + kOffBar);
  x.lead0 = map_to_rank(x.bar0, 0);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + kOffTslot);
  x.abort = reinterpret_cast<volatile int*>(smem + kOffAbort);
  if (x.tid == 0) {
    *x.abort = 0;
    reinterpret_cast<int*>(smem + kOffIssued)[0] = -1;
    reinterpret_cast<int*>(smem + kOffIssued)[1] = -1;
    for (int i = 0; i < kKRing; ++i) {
      mbar_init(x.bar(kKFull + i), 1);
      mbar_init(x.bar(kKEmpty + i), 1);
      mbar_init(x.bar(kPeerK + i), 1);
    }
    for (int i = 0; i < kVRing; ++i) {
      mbar_init(x.bar(kVFull + i), 1);
      mbar_init(x.bar(kVEmpty + i), 1);
      mbar_init(x.bar(kPeerV + i), 1);
    }
    mbar_init(x.bar(kQFull), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(x.bar(kSFull + i), 2);  // Q K^T and the key scales
      mbar_init(x.bar(kSFree + i), 2 * kGroupWarps);
      mbar_init(x.bar(kPFull + i), 2 * kGroupWarps);
      mbar_init(x.bar(kOReady + i), kGroupWarps);
      mbar_init(x.bar(kScFree + i), kGroupWarps);
      mbar_init(x.bar(kXL + i), 8);
    }
    for (int i = 0; i < 8; ++i) mbar_init(x.bar(kX + i), 4);
    mbar_init(x.bar(kDrainQK), 1);
    mbar_init(x.bar(kDrainPV), 1);
    fence_barrier_init();
  }
  if (x.warp == 1) pair_alloc(smem_u32(tslot), kTmemCols);
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // the barriers of both CTAs are there
  fence_after_sync();
  x.tbase = *tslot;

  if (x.n_chunks > 0) {
    if (x.tid == 0) {  // this CTA's rows of q (rows past the last are zeros)
      tma_prefetch_desc(&maps.q);
      mbar_arrive_expect_tx(x.bar(kQFull), kKSlot);
      const int qrow = x.tok0 * x.H + x.row0 + kOwnRows * x.rank;
      for (int j = 0; j < 4; ++j)
        tma_load_2d(smem_u32(smem + kOffQ + j * kBox), &maps.q, 128 * j, qrow, x.bar(kQFull));
      tma_load_2d(smem_u32(smem + kOffQ + 4 * kBox), &maps.qr, kRank, qrow, x.bar(kQFull));
    }
    __syncwarp();
  }
  if (x.warp >= 4) {
    softmax_rows<SCALE>(x, maps, p);
  } else if (x.n_chunks > 0) {
    if (x.warp == 0) {
      load_boxes<BOX>(x, maps, p);
    } else if (x.warp == 2) {
      prepare_keys<BOX, SCALE>(x, p);
    } else if (x.warp == 1) {
      if (x.rank == 0) qk_issue(x);
      else pass_keys(x);
    } else {
      if (x.rank == 0) pv_issue(x);
      else pass_values(x);
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  // every load must have landed before the CTA exits (all were consumed unless a
  // wait gave up): the last one issued to each slot
  if (x.tid == 0 && x.n_chunks > 0) {
    const volatile int* issued = reinterpret_cast<const volatile int*>(smem + kOffIssued);
    for (int i = 0; i < kKRing && issued[0] - i >= 0; ++i)
      drain_wait(x, x.bar(kKFull + (issued[0] - i) % kKRing), ((issued[0] - i) / kKRing) & 1, 13);
    for (int i = 0; i < kVRing && issued[1] - i >= 0; ++i)
      drain_wait(x, x.bar(kVFull + (issued[1] - i) % kVRing), ((issued[1] - i) / kVRing) & 1, 14);
    drain_wait(x, x.bar(kQFull), 0, 15);
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // the pair's instructions and arrivals are done in both CTAs
  fence_after_sync();
  if (x.warp == 1) pair_dealloc(x.tbase, kTmemCols);
}

template <int BOX, Scale SCALE>
cudaError_t launch_variant(const PairMaps& maps, const DecodeParams& p, unsigned items, int* status,
                           cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(decode_pair_kernel<BOX, SCALE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2u * items);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_pair_kernel<BOX, SCALE>, maps, p, status);
}

template <int BOX>
cudaError_t launch_box(const PairMaps& maps, const DecodeParams& p, unsigned items, int* status, cudaStream_t stream) {
  if (p.kv_scales == nullptr) return launch_variant<BOX, Scale::kNone>(maps, p, items, status, stream);
  if (p.scale_group % kUni == 0) return launch_variant<BOX, Scale::kSixteen>(maps, p, items, status, stream);
  return launch_variant<BOX, Scale::kKey>(maps, p, items, status, stream);
}

}  // namespace

cudaError_t launch_decode_pair(const DecodeParams& p, int64_t q_rows, int64_t kv_rows, unsigned items, int* status,
                               cudaStream_t stream) {
  if (p.block_size % 16 != 0 || p.items == nullptr) return cudaErrorInvalidValue;
  // the highest box that never crosses a block's end
  const int box = p.block_size % 64 == 0 ? 64 : p.block_size % 32 == 0 ? 32 : 16;
  PairMaps maps{};
  cudaError_t e = make_row_map(&maps.q, p.q, static_cast<uint64_t>(q_rows), kOwnRows, true);
  if (e == cudaSuccess) e = make_row_map(&maps.qr, p.q, static_cast<uint64_t>(q_rows), kOwnRows, true, 64);
  if (e == cudaSuccess) e = make_row_map(&maps.kv, p.kv, static_cast<uint64_t>(kv_rows), box, true);
  if (e == cudaSuccess) e = make_row_map(&maps.kvr, p.kv, static_cast<uint64_t>(kv_rows), box, true, 64);
  if (e == cudaSuccess) e = make_out_map(&maps.out, p.out, static_cast<uint64_t>(q_rows), 1, true, 64, 32, true);
  if (e == cudaSuccess)
    e = make_out_map(&maps.part, p.segm_out, static_cast<uint64_t>(p.segm_rows), 1, false, 32, 32, true);
  if (e != cudaSuccess) return e;
  return box == 64 ? launch_box<64>(maps, p, items, status, stream)
         : box == 32 ? launch_box<32>(maps, p, items, status, stream)
                     : launch_box<16>(maps, p, items, status, stream);
}

}  // namespace mla

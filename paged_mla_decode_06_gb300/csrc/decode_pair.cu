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
// That is 1860 tensor cycles a chunk and pair. An instruction reads the same
// shared-memory offsets in both CTAs, so a CTA's own keys as B of Q K^T and its
// columns as B of P V cannot share a copy: K and V have rings of their own, and
// a chunk brings 68 KB into each SM, 36 of keys and 32 of values.
//
// Measured: 2190 cycles a chunk where tiles follow one another: 68 of the 88 us that
// the kernel takes for 64 requests over 8192 common keys at 128 heads (165 GFLOP, 62 chunks a
// pair; 0.99 of the measured bf16 rate, half of the e4m3 one). What bounds it there is the
// tensor pipe, 85 % busy, and a softmax of about 4400 cycles a chunk for each of its
// two groups, which leaves no slack. The rest of the time is the start (6 us to the
// first P V) and the items' ends (5 us each: the last P V, the output, the first scores of
// the next). The value-split kernel, which computes all scores in both SMs and the
// softmax of all 128 rows too, takes 3100 to 3400 cycles a chunk.
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
// Warps: 0 loads q and keys, 1 issues Q K^T (rank 1: passes keys on), 2 prepares the
// keys' scales, 3 issues P V (passes values on), 4 and 5 load values, 6 watches the
// time, 8-23 softmax and epilogue (7 has no work: registers move by four warps). 80
// registers a thread at launch; the softmax spills 68 to 88 bytes (32 without group scales).
// Every wait is bounded: a timeout records a code in the status word, stops
// the CTA's work, drains what was issued and exits.
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
constexpr int kRoleWarps = 8;             // warps 0-7, then the softmax's
constexpr int kThreads = 32 * (kRoleWarps + kSoftWarps);
// Registers a thread: the launch's (of 65536, a warp's in steps of 8 a thread), and after the roles
// have given some of theirs up for the softmax; the sum stays within the launch's.
constexpr int kLaunchRegs = 80, kRoleRegs = 40, kSoftRegs = 96;
static_assert(kThreads * kLaunchRegs <= 65536 &&
                  32 * (kRoleWarps * kRoleRegs + kSoftWarps * kSoftRegs) <= kThreads * kLaunchRegs,
              "registers of the launch");
constexpr int kPTile = kOwnRows * kKeys;  // one term of P of a chunk
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;            // 256 columns: 128 for each j
constexpr uint32_t kTmemS = 256;          // [2] 64: S of chunk c at c % 2
constexpr uint64_t kDefaultWaitNs = 2000000000ull;
constexpr uint32_t kSleepNs = 20000;
// 2^kPBias is the weight of the reference, 2^(kPBias + kMove) the largest. (Of 0 to 4, which
// move 11.75 to 7.75: 2 to 4 % of the time; 4 keeps 7 bits of a weight furthest down.)
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
  kSFull,                      // [2] (of chunk c at c % 2, as the next four) S written and key scales ready
  kSFree = kSFull + 2,         // [2] rank 0: S read by both CTAs
  kPFull = kSFree + 2,         // [2] rank 0: P written by both CTAs, O_0 rescaled
  kOReady = kPFull + 2,        // [2] rank 0: O_1 rescaled
  kX = kOReady + 2,            // [4][2] (at c % 4) the four warps of 32 rows have posted their maxima
  kScFree = kX + 8,            // [2] key scales read
  kXL = kScFree + 2,           // [2] the eight warps of 32 rows have posted their sums of an item
  kOFree = kXL + 2,            // rank 0: both CTAs have read O of an item
  kStage,                      // [2] the output of an item with keys, number m at m % 2, has left the value ring
  kDrainQK = kStage + 2,       // Q K^T and P V complete, in both CTAs
  kDrainPV,
  kDone,                       // all softmax warps have ended
  kNumBars
};

// Shared memory.
constexpr int kOffBar = 0;
constexpr int kOffWatch = 400;                  // Watch
constexpr int kOffTslot = 448;
constexpr int kOffIssued = 464;                  // {last chunk of keys, of values j = 0, 1, last q} issued
constexpr int kOffMask = 480;                    // [2][4] bits of existing keys of chunk c (at c % 2)
constexpr int kOffXMax = 512;                    // [4][4][64] maxima of chunk c (at c % 4) by key quarter
constexpr int kOffScale = kOffXMax + 4096;       // [2][mul, add, inv][128]
constexpr int kOffLsum = kOffScale + 3 * 1024;   // [2][2][4][64] row sums (of item i at i % 2) by group and key quarter
constexpr int kOffQ = 12288;                     // 4 boxes of 64 rows, 128-byte swizzle; rope box, 64-byte swizzle
constexpr int kOffP = kOffQ + kKSlot;            // [c % 2][hi, lo] 64 rows x 128 keys, 128-byte swizzle
constexpr int kOffK = kOffP + 4 * kPTile;
constexpr int kOffV = kOffK + kKRing * kKSlot;
constexpr int kSmem = kOffV + kVRing * kVSlot + 1024;  // + alignment slack
static_assert(kNumBars * 8 <= kOffWatch && kOffLsum + 4096 <= kOffQ, "header space");
static_assert(kSmem <= 232448, "shared memory budget");
static_assert(kVRing * kVSlot == kSoftWarps * 4096, "a group stages its output in the slots of its chunks");

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
  uint32_t tbase;
  int tid, warp, lane, rank;
  int first, last;       // the pair's items
  __device__ uint32_t bar(int i) const { return bar0 + 8u * i; }
  __device__ uint32_t lead(int i) const { return lead0 + 8u * i; }
};

// An item of the list.
struct Item {
  int unit, row0, seg_start, seg_end, n;  // n: chunks
  int pslot;             // first row of the partial's slot, -1: write out/lse
  int tok0, tokens;
  int see0;              // keys that the first token of the unit sees; INT_MAX: all rows see all keys
};
// Whether one of the softmax's groups writes the output of an item that others follow, while
// the other goes on: of many rows, whose stores take their time however many warps
// make them (64 requests over 8192 common keys, 128 heads: 102.4 -> 99.7 us). Few rows are
// done sooner by both (16 heads over 16384 common keys: 52.9 -> 51.1).
__device__ __forceinline__ bool one_writes(const Item& it, int num_heads) {
  return it.tokens * num_heads - it.row0 > kOwnRows;
}
// The same for the whole warp, and for the compiler: loops that it takes for
// divergent keep the matrix instructions' descriptors in vector registers (250
// cycles an instruction).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ Item item_at(const DecodeParams& p, int i) {
  int4 a = reinterpret_cast<const int4*>(p.items)[2 * i];
  int4 b = reinterpret_cast<const int4*>(p.items)[2 * i + 1];
  a = make_int4(uniform(a.x), uniform(a.y), uniform(a.z), uniform(a.w));
  b = make_int4(uniform(b.x), uniform(b.y), uniform(b.z), uniform(b.w));
  return Item{a.x, a.y * kRows, a.z, a.w, a.w > a.z ? cdiv(a.w - a.z, kKeys) : 0, b.x, b.y, b.z & kItemTokens,
              (b.z & kItemPrefix) != 0 ? INT_MAX : b.w};
}

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
// The matrix instructions of a step, with descriptors formed by additions to
// their lower words from a base in between: what changes from one instruction to
// the next is two words. (64-bit descriptors computed outside took the issuing
// warp 100 to 125 cycles an instruction, more than its 64 tensor cycles.)
//
// Four steps of 32 columns of a 128-byte column box: D (+)= A B.
__device__ __forceinline__ void mma_box(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b32 l, t;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n"
      " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p;\n"
      " add.u32 t, %1, 2;\n add.u32 l, %3, 2;\n mov.b64 a, {t, %2};\n mov.b64 b, {l, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, 1;\n"
      " add.u32 t, %1, 4;\n add.u32 l, %3, 4;\n mov.b64 a, {t, %2};\n mov.b64 b, {l, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, 1;\n"
      " add.u32 t, %1, 6;\n add.u32 l, %3, 6;\n mov.b64 a, {t, %2};\n mov.b64 b, {l, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, 1;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Two steps of the 64-byte rope box: D += A B.
__device__ __forceinline__ void mma_rope(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                         uint32_t idesc) {
  asm volatile(
      "{\n .reg .b32 l, t;\n .reg .b64 a, b;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, 1;\n"
      " add.u32 t, %1, 2;\n add.u32 l, %3, 2;\n mov.b64 a, {t, %2};\n mov.b64 b, {l, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, 1;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc)
      : "memory");
}
// A step of 32 keys of P V, both terms of P (kPTile bytes apart): D (+)= A B, D += A' B.
__device__ __forceinline__ void mma_terms(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                          uint32_t id_hi, uint32_t id_lo, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b32 t;\n .reg .b64 a, b;\n setp.ne.b32 p, %7, 0;\n"
      " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p;\n"
      " add.u32 t, %1, %8;\n mov.b64 a, {t, %2};\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %6, 1;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(id_hi), "r"(id_lo), "r"(accumulate), "n"(kPTile >> 4)
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
// A wait ends when its phase completes or when the CTA gives up, which one warp
// decides for all (watch): a clock, a limit and a report at each of some thirty waits
// made the kernel's code a third larger, and the warps waited for instructions a
// fifth of their time.
struct Watch {
  int* status;
  uint64_t ns;            // limit
  volatile int abort;
  volatile int progress;  // changes with every chunk of the softmax
};
__device__ __forceinline__ Watch* watch_of(const uint8_t* smem) {
  return reinterpret_cast<Watch*>(const_cast<uint8_t*>(smem) + kOffWatch);
}

// Wait on a barrier phase, sleeping; false when the CTA gives up. Barriers that the
// other CTA arrives on are waited for as the CTA's own: no thread reads what one of
// the other CTA wrote through the generic proxy (P, S and O are read by the tensor
// core of the SM that holds them, after proxy and tcgen05 fences), and acquire and
// release at cluster scope took 1000 to 2000 cycles each (168 us against 133 for 64
// requests over 8192 common keys, 128 heads).
__device__ __forceinline__ bool warp_wait(const Ctx& x, uint32_t bar, uint32_t parity) {
  bool ok = mbar_test_wait(bar, parity);
  while (!__all_sync(0xffffffffu, ok)) {
    ok = mbar_try_wait_sleep(bar, parity, kSleepNs);
    if (__any_sync(0xffffffffu, !ok && watch_of(x.smem)->abort != 0)) return false;
  }
  return true;
}
// Warp 6: gives up, with a code in the status word, when the softmax has made no
// progress for the limit. All other waits come to an end with the softmax's, or
// are bounded by themselves (drain_wait). (It sleeps on the barrier that ends its
// work: asleep on a timer it kept the CTA for 1 to 2 us more.)
__device__ void watch(const Ctx& x) {
  Watch* w = watch_of(x.smem);
  int seen = -1;
  uint64_t t0 = 0;
  if (x.lane == 0) {
    while (!mbar_try_wait_sleep(x.bar(kDone), 0, kSleepNs) && !w->abort) {
      const uint64_t now = global_timer_ns();
      if (w->progress != seen) {
        seen = w->progress;
        t0 = now;
      } else if (now - t0 > w->ns) {
        if (w->status != nullptr) atomicCAS(w->status, 0, 11);
        w->abort = 1;
      }
    }
  }
  __syncwarp();
}
// Wait that ignores the abort flag (teardown), bounded by itself.
__device__ __forceinline__ void drain_wait(const Ctx& x, uint32_t bar, uint32_t parity, int code) {
  if (mbar_test_wait(bar, parity)) return;  // (nearly always; reading the timer takes longer)
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_sleep(bar, parity, kSleepNs)) {
    if (global_timer_ns() - t0 > kDefaultWaitNs) {
      if (watch_of(x.smem)->status != nullptr) atomicCAS(watch_of(x.smem)->status, 0, code);
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
  __device__ __forceinline__ int look(const Ctx& x, const DecodeParams& p, const Item& it, int w0) const {
    const int pos = it.seg_start + w0 * kKeys + x.lane * BOX;
    if (pos >= it.seg_end) return -BOX;
    const int blk = pos / p.block_size;
    const int b = p.block_table[static_cast<int64_t>(it.unit) * p.bt_stride + blk];
    return b < 0 ? -BOX : b * p.block_size + (pos - blk * p.block_size);
  }
  __device__ __forceinline__ void start(const Ctx& x, const DecodeParams& p, const Item& it) {
    cur = look(x, p, it, 0);
    nxt = look(x, p, it, kSpan);
  }
  // moves on to the window of chunk c (called for every chunk in turn)
  __device__ __forceinline__ void at(const Ctx& x, const DecodeParams& p, const Item& it, int c) {
    if (c > 0 && c % kSpan == 0) {
      cur = nxt;
      nxt = look(x, p, it, c + kSpan);
    }
  }
  __device__ __forceinline__ int row(int c, int run) const {
    return __shfl_sync(0xffffffffu, cur, kPer * (c % kSpan) + run);
  }
};

// Warp 0: q of each item (its 64 rows), and the keys of each chunk (five column
// boxes of this CTA's 64 rows), a box by each of as many lanes. Warps 4 and 5: one
// column box of values of each chunk (all 128 rows). Copies of one warp move about 27
// bytes a clock, of the 36 that a chunk needs in 1860 cycles, and a warp of its
// own runs some hundred instructions in that time: with keys and values in one
// warp a chunk took 2300 to 3500 cycles, with values and scales in one 4700. The
// rings run on across items: q and the first keys of the next one load while this
// one's last chunks and its output are under way, and so do the values of its first
// chunk; those of the second wait for the output, which is staged in the slots of this one's
// last chunk.
template <int BOX>
__device__ void load_keys(const Ctx& x, const PairMaps& maps, const DecodeParams& p) {
  constexpr int kSub = kHalf / BOX;  // boxes high of 64 rows
  const int box = x.lane / kSub, run = x.lane % kSub;
  volatile int* issued = reinterpret_cast<volatile int*>(x.smem + kOffIssued);
  const uint32_t base = smem_u32(x.smem);
  RowWindow<BOX> w;
  int c = 0, q = 0;  // chunks and q's so far
  for (int i = x.first; i < x.last; ++i) {
    const Item it = item_at(p, i);
    if (it.n == 0) continue;
    w.start(x, p, it);
    for (int k = 0; k < it.n; ++k, ++c) {
      const int s = c % kKRing;
      if (c >= kKRing && !warp_wait(x, x.bar(kKEmpty + s), (c / kKRing - 1) & 1)) return;
      // (q, once Q K^T of the item before is complete)
      if (k == 0 && c > 0 && !warp_wait(x, x.bar(kKEmpty + (c - 1) % kKRing), ((c - 1) / kKRing) & 1)) return;
      w.at(x, p, it, k);
      const uint32_t full = x.bar(kKFull + s), to = base + kOffK + s * kKSlot;
      if (x.lane == 0) {
        mbar_arrive_expect_tx(full, kKSlot);
        issued[0] = c;
        if (k == 0) {
          mbar_arrive_expect_tx(x.bar(kQFull), kKSlot);
          issued[3] = q;
        }
      }
      __syncwarp();
      if (k == 0 && x.lane < 5) {  // (rows past the last are zeros)
        const int qrow = it.tok0 * p.num_heads + it.row0 + kOwnRows * x.rank;
        tma_load_2d(base + kOffQ + x.lane * kBox, x.lane < 4 ? &maps.q : &maps.qr, 128 * x.lane, qrow, x.bar(kQFull));
      }
      const int row = w.row(k, x.rank * kSub + run);
      if (box < 5)
        tma_load_2d(to + box * kBox + run * BOX * (box < 4 ? 128 : 64), box < 4 ? &maps.kv : &maps.kvr, 128 * box, row, full);
      __syncwarp();
    }
    ++q;
  }
}

template <int BOX>
__device__ void load_values(const Ctx& x, const PairMaps& maps, const DecodeParams& p, int j) {
  constexpr int kRuns = kKeys / BOX;  // boxes high of 128 rows
  volatile int* issued = reinterpret_cast<volatile int*>(x.smem + kOffIssued);
  const int run = x.lane % kRuns;
  const uint32_t to0 = smem_u32(x.smem) + kOffV + run * BOX * 128;
  RowWindow<BOX> w;
  int c = 0, m = 0;   // chunks, items with keys so far
  bool half = false;  // the last one's output takes half of the ring
  for (int i = x.first; i < x.last; ++i) {
    const Item it = item_at(p, i);
    if (it.n == 0) continue;
    w.start(x, p, it);
    for (int k = 0; k < it.n; ++k, ++c) {
      const int v = 2 * c + j, s = v % kVRing;
      // The output one item back is staged in all slots or in those of its last chunk, which
      // are the second one's here; the one before may have been in the first one's. (The
      // barriers' next phases wait for this item's values: none is passed over.)
      const int out = k == 0 && half ? m - 2 : m - 1;
      if (k < 2 && out >= 0 && !warp_wait(x, x.bar(kStage + (out & 1)), (out >> 1) & 1)) return;
      w.at(x, p, it, k);
      const int row = w.row(k, run);
      if (v >= kVRing && !warp_wait(x, x.bar(kVEmpty + s), (v / kVRing - 1) & 1)) return;
      if (x.lane == 0) {
        mbar_arrive_expect_tx(x.bar(kVFull + s), kVSlot);
        issued[1 + j] = c;
      }
      __syncwarp();
      if (x.lane < kRuns) tma_load_2d(to0 + s * kVSlot, &maps.kv, 128 * (2 * j + x.rank), row, x.bar(kVFull + s));
      __syncwarp();
    }
    ++m;
    half = one_writes(it, p.num_heads);
  }
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
  constexpr int kParts = SCALE == Scale::kKey ? 4 : 1;
  const int lane = x.lane;
  RowWindow<BOX> w;
  float sc[kParts];
  uint32_t bits = 0u;  // lane k < 4: existing keys of part k
  int g = 0;           // chunks so far
  for (int i = x.first; i < x.last; ++i) {
    const Item it = item_at(p, i);
    if (it.n == 0) continue;
    w.start(x, p, it);
    auto read = [&](int c) {
      w.at(x, p, it, c);
      const int n = it.seg_end - (it.seg_start + c * kKeys);
      // whether a run of this chunk has no block
      const uint32_t gone = __ballot_sync(0xffffffffu, w.cur < 0) >> (RowWindow<BOX>::kPer * (c % RowWindow<BOX>::kSpan));
      const bool whole = n >= kKeys && (gone & ((1u << RowWindow<BOX>::kPer) - 1u)) == 0u;
      bits = 0xffffffffu;
      if (!whole) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = 32 * k + lane;
          const int row = w.row(c, j / BOX);  // (all lanes: a shuffle)
          const uint32_t there = __ballot_sync(0xffffffffu, j < n && row >= 0);
          if (lane == k) bits = there;
        }
      }
      if constexpr (SCALE != Scale::kNone) {
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          const int j = SCALE == Scale::kKey ? 32 * k + lane : kUni * (lane & 7);
          const int row = w.row(c, j / BOX);
          sc[k] = j < n && row >= 0 ? scale_of_slot(p, row + j % BOX) : 1.f;
        }
      }
    };
    read(0);
    for (int c = 0; c < it.n; ++c, ++g) {
      const int b = g & 1;
      if (g >= 2 && !warp_wait(x, x.bar(kScFree + b), ((g >> 1) - 1) & 1)) return;
      float* ks = reinterpret_cast<float*>(x.smem + kOffScale) + b * 3 * kKeys;
      if (lane < 4) reinterpret_cast<uint32_t*>(x.smem + kOffMask)[b * 4 + lane] = bits;
      if constexpr (SCALE != Scale::kNone) {
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          const KeyScale ks1 = key_scale(sc[k], p.score_scale_log2);
          const int at = SCALE == Scale::kKey ? 32 * k + lane : kUni * lane;
          if (SCALE == Scale::kKey || lane < kKeys / kUni) {
            ks[at] = ks1.mul;
            ks[kKeys + at] = ks1.add;
            ks[2 * kKeys + at] = ks1.inv;
          }
        }
      }
      __syncwarp();
      if (g >= 2 && !warp_wait(x, x.bar(kSFull + b), ((g >> 1) - 1) & 1)) return;  // S two chunks back
      if (lane == 0) mbar_arrive(x.bar(kSFull + b));
      if (c + 1 < it.n) read(c + 1);
    }
  }
}

// ------------------------------------------------------------------ MMA issue
__device__ __forceinline__ uint32_t lo(uint64_t v) { return static_cast<uint32_t>(v); }
__device__ __forceinline__ uint32_t hi(uint64_t v) { return static_cast<uint32_t>(v >> 32); }

// Rank 0, warp 1.
__device__ void qk_issue(const Ctx& x, const DecodeParams& p) {
  constexpr uint32_t kId = instr_desc(kRows, kKeys, 0, 0, false, false);
  const uint32_t base = smem_u32(x.smem);
  const uint64_t q_desc = smem_desc_sw128(base + kOffQ, 16, 1024);
  const uint64_t qr_desc = smem_desc_sw64(base + kOffQ + 4 * kBox, 512);
  const uint64_t k_desc = smem_desc_sw128(base + kOffK, 16, 1024);
  const uint64_t kr_desc = smem_desc_sw64(base + kOffK + 4 * kBox, 512);
  const bool one = elect_one();
  bool ok = true;
  int c = 0, q = 0;  // chunks, q's so far
  for (int i = x.first; i < x.last && ok; ++i) {
    const int n = item_at(p, i).n;
    if (n > 0) ok = warp_wait(x, x.bar(kQFull), q++ & 1);
    for (const int end = c + n; c < end && ok; ++c) {
      const int b = c & 1, s = c % kKRing;
      ok = warp_wait(x, x.bar(kKFull + s), (c / kKRing) & 1) &&
           warp_wait(x, x.bar(kPeerK + s), (c / kKRing) & 1) &&
           (c < 2 || warp_wait(x, x.bar(kSFree + b), ((c >> 1) - 1) & 1));
      if (!ok) break;
      fence_after_sync();
      const uint32_t at = (s * kKSlot) >> 4;
      const uint32_t d = x.tbase + kTmemS + 64u * b;
      if (one) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mma_box(d, lo(q_desc) + (i * kBox >> 4), hi(q_desc), lo(k_desc) + at + (i * kBox >> 4), hi(k_desc), kId,
                  i != 0 ? 1u : 0u);
        mma_rope(d, lo(qr_desc), hi(qr_desc), lo(kr_desc) + at, hi(kr_desc), kId);
        pair_commit(x.bar(kSFull + b));
        pair_commit(x.bar(kKEmpty + s));
      }
      __syncwarp();
    }
  }
  if (one) {
    pair_commit(x.bar(kDrainQK));
    drain_wait(x, x.bar(kDrainQK), 0, 25);
  }
  __syncwarp();
}

// Rank 0, warp 3: P V of a chunk by halves of the columns, so that a half of O may
// be rescaled while the other is multiplied.
__device__ void pv_issue(const Ctx& x, const DecodeParams& p) {
  constexpr uint32_t kIdHi = instr_desc(kRows, 256, 1, 0, false, true);
  constexpr uint32_t kIdLo = instr_desc(kRows, 256, 0, 0, false, true);
  const uint32_t base = smem_u32(x.smem);
  const uint64_t v_desc = smem_desc_sw128(base + kOffV, kBox, 1024);  // MN-major
  const uint64_t p_desc = smem_desc_sw128(base + kOffP, 16, 1024);
  const bool one = elect_one();
  bool ok = true;
  int g = 0, outs = 0;  // boxes, outputs with keys so far
  for (int i = x.first; i < x.last && ok; ++i) {
    const int n = item_at(p, i).n;
    // O of the item before has been read
    if (n > 0 && outs++ > 0) ok = warp_wait(x, x.bar(kOFree), outs & 1);
    const int begin = g;
    for (const int end = g + 2 * n; g < end && ok; ++g) {
      const int j = g & 1, c = g >> 1, b = c & 1, s = g % kVRing;
      ok = warp_wait(x, x.bar((j == 0 ? kPFull : kOReady) + b), (c >> 1) & 1) &&
           warp_wait(x, x.bar(kVFull + s), (g / kVRing) & 1) &&
           warp_wait(x, x.bar(kPeerV + s), (g / kVRing) & 1);
      if (!ok) break;
      fence_after_sync();
      const uint32_t vb = lo(v_desc) + ((s * kVSlot) >> 4), pb = lo(p_desc) + ((b * 2 * kPTile) >> 4);
      const uint32_t d = x.tbase + kTmemO + 128u * j;
      const uint32_t more = g - begin > 1 ? 1u : 0u;
      if (one) {
#pragma unroll
        for (int ks = 0; ks < kKeys / 32; ++ks)
          mma_terms(d, pb + (ks * 32 >> 4), hi(p_desc), vb + (ks * 32 * 128 >> 4), hi(v_desc), kIdHi, kIdLo,
                    ks != 0 ? 1u : more);
        pair_commit(x.bar(kVEmpty + s));
      }
      __syncwarp();
    }
  }
  if (one) {
    pair_commit(x.bar(kDrainPV));
    drain_wait(x, x.bar(kDrainPV), 0, 29);
  }
  __syncwarp();
}

// Rank 1, warps 1 and 3: what has landed here, passed on to rank 0.
__device__ void pass_keys(const Ctx& x, const DecodeParams& p) {
  bool ok = true;
  int c = 0, q = 0;
  for (int i = x.first; i < x.last && ok; ++i) {
    const int n = item_at(p, i).n;
    if (n > 0) ok = warp_wait(x, x.bar(kQFull), q++ & 1);  // (before the item's first keys)
    for (const int end = c + n; c < end && ok; ++c) {
      const int s = c % kKRing;
      ok = warp_wait(x, x.bar(kKFull + s), (c / kKRing) & 1);
      if (ok && x.lane == 0) mbar_arrive_remote(x.lead(kPeerK + s));
      __syncwarp();
    }
  }
  if (x.lane == 0) drain_wait(x, x.bar(kDrainQK), 0, 25);
  __syncwarp();
}
__device__ void pass_values(const Ctx& x, const DecodeParams& p) {
  bool ok = true;
  int g = 0;
  for (int i = x.first; i < x.last && ok; ++i) {
    for (const int end = g + 2 * item_at(p, i).n; g < end && ok; ++g) {
      const int s = g % kVRing;
      ok = warp_wait(x, x.bar(kVFull + s), (g / kVRing) & 1);
      if (ok && x.lane == 0) mbar_arrive_remote(x.lead(kPeerV + s));
      __syncwarp();
    }
  }
  if (x.lane == 0) drain_wait(x, x.bar(kDrainPV), 0, 29);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax + epilogue
template <Scale SCALE>
__device__ void softmax_rows(const Ctx& x, const PairMaps& maps, const DecodeParams& p) {
  constexpr bool UNI = SCALE == Scale::kSixteen, ONE = SCALE == Scale::kNone;
  const int lane = x.lane;
  const int sw = x.warp - kRoleWarps;
  const int q4 = x.warp & 3;               // TMEM lane quarter of this warp
  const int rq = q4 & 1;                   // its 32 of the CTA's 64 rows
  const int kq = q4 >> 1;                  // its half of a chunk's keys
  const int h = sw >> 3;                   // chunks c with c % 2 == h, and buffer
  const int kh = (sw >> 2) & 1;            // its 32 keys of the half
  const int part = 2 * kq + kh;            // key quarter (and, of a rescaling, columns of O_kh)
  const int r = rq * 32 + lane;            // row within the CTA
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const int H = p.num_heads;
  bool ok = true;

  float* xmax = reinterpret_cast<float*>(x.smem + kOffXMax) + r;
  uint8_t* prow = x.smem + kOffP + h * 2 * kPTile + r * 128;
  const int c0 = ((2 * part) ^ (r & 7)) << 4, c1 = ((2 * part + 1) ^ (r & 7)) << 4;
  const uint32_t ts = x.tbase + lane_off + kTmemS + 64u * h + kPart * kh;

  auto pv_done = [&](int c, int j) {
    const int g = 2 * c + j;
    return warp_wait(x, x.bar(kVEmpty + g % kVRing), (g / kVRing) & 1);
  };
  int first = 0;  // chunks (of all items) before this item's: buffers and phases run on
  int m = 0;      // items with keys so far
  for (int i = x.first; i < x.last; ++i) {
    const Item it = item_at(p, i);
    const int n = it.n, end = first + n;
    const int rows_total = it.tokens * H;
    const int rho = it.row0 + kOwnRows * x.rank + r;  // row within the unit
    const bool row_ok = rho < rows_total;
    const int token = rho / H;
    const int vis = !row_ok ? 0 : (it.see0 == INT_MAX ? INT_MAX : it.see0 + token);
    // keys from here on (of chunk 0 of all items' chunks) are not seen by all rows
    const int start = it.seg_start - first * kKeys;
    const int all_see = it.see0 == INT_MAX ? INT_MAX : it.see0 + it.row0 / H - start;
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
    // before it posts its own of c + 3, which the other waits for before it posts
    // that of c + 4: neither the barrier's phase nor the four buffers are passed over.
    auto follow_other = [&](int c) {
      if (!warp_wait(x, x.bar(kX + 2 * (c & 3) + rq), (c >> 2) & 1)) return false;
      follow(row_max(c));
      return true;
    };
    for (int c = first + ((first & 1) ^ h); c < end; c += 2) {
      const int ph = (c >> 1) & 1;
      ok = warp_wait(x, x.bar(kSFull + h), ph);
      if (!ok) break;
      if (sw == 0 || sw == 8) watch_of(x.smem)->progress = c;
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
      const int lim = min(vis, it.seg_end) - (start + c * kKeys + kPart * part);
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
      xmax[((c & 3) * 4 + part) * kOwnRows] = fmaxf(m[0], m[1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(x.bar(kX + 2 * (c & 3) + rq));
      ok = c == first || follow_other(c - 1);
      if (!ok) break;
      ok = warp_wait(x, x.bar(kX + 2 * (c & 3) + rq), (c >> 2) & 1);
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
      ok = c < 2 || pv_done(c - 2, 1);
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
          ok = warp_wait(x, x.bar(kVFull + g % kVRing), (g / kVRing) & 1);  // (its writes are seen here too)
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
        ok = pv_done(c - 1, kh);
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

    if (!ok) break;
    // ---------------------------------------------------------------- epilogue
    // The group of the last chunk writes the output, while the other goes on to
    // the next item's first chunk, which is its own: P V over that waits for O alone.
    // After the last item, and of few rows, both write.
    const bool mine = h == ((end - 1) & 1), both = i + 1 == x.last || !one_writes(it, H);
    if (n > 0 && !mine) ok = follow_other(end - 1);
    // (all sums of the item before are there: no arrival counts for another's phase)
    if (ok && i > x.first) ok = warp_wait(x, x.bar(kXL + rq), (i - 1 - x.first) & 1);
    if (!ok) break;
    float* lsum = reinterpret_cast<float*>(x.smem + kOffLsum) + ((i - x.first) & 1) * 8 * kOwnRows + r;
    lsum[(4 * h + part) * kOwnRows] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kXL + rq));
    first = end;
    m += n > 0 ? 1 : 0;
    if (!mine && !both) continue;
    ok = warp_wait(x, x.bar(kXL + rq), (i - x.first) & 1);
    // O is complete with the last chunk
    if (ok && n > 0) ok = pv_done(end - 1, 1);
    if (!ok) break;
    fence_after_sync();
    const bool fin = it.pslot < 0;
    float mult = 0.f;
    if (row_ok) {
      float L = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) L += lsum[k * kOwnRows];
      const float base = ref == -INFINITY ? 0.f : ref - kPBias;  // the reference of O and the sum
      const int head = rho - token * H;
      const int64_t th = static_cast<int64_t>(it.tok0) * H + rho;
      const bool writes = mine && kq == 0 && kh == 0;
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
          const int64_t at = static_cast<int64_t>(it.pslot) + kOwnRows * x.rank + r;
          const float2 ms = partial_sums(L > 0.f ? base : -INFINITY, L);
          p.segm_max[at] = ms.x;
          p.segm_expsum[at] = ms.y;
        }
      }
      mult *= p.kv_scale;
    }
    // Each warp scales its 32 rows of 64 columns (of 128, where one group writes) and
    // stages them, 128 bytes of each row at a time, in the 128-byte swizzle, in its
    // 4 KB of the value ring (its group's half, the slots of the last chunk, which P V has
    // read and whose next values wait for kStage), and one TMA tensor store writes each
    // staged tile. Where some of the 32 rows do not exist the warp stores the others, four at
    // a time (a row by each lane: 1400 cycles a tile of 16), and the zeros of an
    // item without keys, which has no slots. (TMEM loads are warp-collective.)
    const int wr = it.row0 + kOwnRows * x.rank + 32 * rq;  // the warp's first row within the unit
    if (wr < rows_total) {
      const bool whole = n > 0 && wr + 32 <= rows_total;
      const int z0 = fin ? it.tok0 * H + wr : it.pslot + (wr - it.row0);
      const CUtensorMap* map = fin ? &maps.out : &maps.part;
      uint8_t* buf = x.smem + kOffV + sw * 4096;
      auto store = [&](const uint32_t (&w)[32], int col) {
        if (n > 0) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
          fence_proxy_async_smem();  // (for the store, and for the loads that come here next)
        }
        if (whole) {
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(map, smem_u32(buf), col, 0, z0);
            bulk_commit_group();
            bulk_wait_read<0>();
          }
        } else {
          __syncwarp();
          uint8_t* dst = (fin ? static_cast<uint8_t*>(p.out) : reinterpret_cast<uint8_t*>(p.segm_out)) +
                         (static_cast<int64_t>(z0) * kRank + col) * (fin ? 2 : 4) + 16 * (lane & 7);
          for (int i = lane >> 3; wr + i < min(rows_total, wr + 32); i += 4) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (n > 0) v = *reinterpret_cast<const uint4*>(buf + i * 128 + (((lane ^ i) & 7) << 4));
            *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(i) * kRank * (fin ? 2 : 4)) = v;
          }
        }
        __syncwarp();
      };
      auto load = [&](int at, uint32_t (&o)[32]) {
        if (n > 0) {
          tmem_ld_32x32b_x32(x.tbase + lane_off + kTmemO + at, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
      };
      // quarters of the TMEM columns of O
      const int cq0 = both ? 2 * h + kh : 2 * kh, cq1 = cq0 + (both ? 1 : 2);
#pragma unroll 1
      for (int cq = cq0; cq < cq1; ++cq) {
        const int col0 = 256 * (cq >> 1) + 128 * kq + 64 * (cq & 1);
        if (fin) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
            load(64 * cq + 32 * c, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * mult, __uint_as_float(o[2 * j + 1]) * mult);
              w[16 * c + j] = *reinterpret_cast<const uint32_t*>(&b);
            }
          }
          store(w, col0);
        } else {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
            load(64 * cq + 32 * c, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * mult);
            store(o, col0 + 32 * c);
          }
        }
      }
    }
    // O has been read (of items with keys, whose next one replaces it), and the
    // staged tiles too
    fence_before_sync();
    __syncwarp();
    if (lane == 0 && n > 0) {
      const int count = both ? 1 : 2;
      mbar_arrive_remote(x.lead(kOFree), count);
      mbar_arrive(x.bar(kStage + ((m - 1) & 1)), count);
    }
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(x.bar(kDone));
}

template <int BOX, Scale SCALE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    decode_pair_kernel(const __grid_constant__ PairMaps maps, const DecodeParams p, int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctx x;
  x.smem = smem;
  x.tid = threadIdx.x;
  x.warp = uniform(x.tid >> 5);
  x.lane = x.tid & 31;
  x.rank = uniform(static_cast<int>(cluster_ctarank()));

  x.bar0 = smem_u32(smem + kOffBar);
  x.lead0 = map_to_rank(x.bar0, 0);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + kOffTslot);
  if (x.tid == 0) {
    Watch* w = watch_of(smem);
    w->status = status;
    w->ns = p.wait_ns != 0 ? p.wait_ns : kDefaultWaitNs;
    w->abort = 0;
    w->progress = 0;
    reinterpret_cast<int*>(smem + kOffIssued)[0] = -1;
    reinterpret_cast<int*>(smem + kOffIssued)[1] = -1;
    reinterpret_cast<int*>(smem + kOffIssued)[2] = -1;
    reinterpret_cast<int*>(smem + kOffIssued)[3] = -1;
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
      mbar_init(x.bar(kStage + i), kSoftWarps);
    }
    for (int i = 0; i < 8; ++i) mbar_init(x.bar(kX + i), 4);
    mbar_init(x.bar(kOFree), 2 * kSoftWarps);  // (one group's warps count twice)
    mbar_init(x.bar(kDrainQK), 1);
    mbar_init(x.bar(kDrainPV), 1);
    mbar_init(x.bar(kDone), kSoftWarps);
    fence_barrier_init();
  }
  if (x.warp == 1) pair_alloc(smem_u32(tslot), kTmemCols);
  if (x.tid == 32 * kRoleWarps) {
    tma_prefetch_desc(&maps.kv);
    tma_prefetch_desc(&maps.kvr);
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.qr);
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // the barriers of both CTAs are there
  fence_after_sync();
  x.tbase = *tslot;
  // the list, once the grid that wrote it has completed (what is above this runs
  // beside it); the merge may launch once every CTA is here
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  // (a pair without items runs through, so that all its waits and commits have their match)
  x.first = uniform(p.worker_first[blockIdx.x >> 1]);
  x.last = uniform(p.worker_first[(blockIdx.x >> 1) + 1]);

  if (x.warp >= kRoleWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    softmax_rows<SCALE>(x, maps, p);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRoleRegs));
    if (x.warp == 0) {
      load_keys<BOX>(x, maps, p);
    } else if (x.warp == 2) {
      prepare_keys<BOX, SCALE>(x, p);
    } else if (x.warp == 4 || x.warp == 5) {
      load_values<BOX>(x, maps, p, x.warp - 4);
    } else if (x.warp == 1) {
      if (x.rank == 0) qk_issue(x, p);
      else pass_keys(x, p);
    } else if (x.warp == 3) {
      if (x.rank == 0) pv_issue(x, p);
      else pass_values(x, p);
    } else if (x.warp == 6) {
      watch(x);
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  __syncthreads();
  // every load must have landed before the CTA exits (all were consumed unless a
  // wait gave up): the last one issued to each slot (known once all warps are
  // here: a phase that another follows cannot be waited for by its parity)
  if (x.tid == 0) {
    const volatile int* issued = reinterpret_cast<const volatile int*>(smem + kOffIssued);
    for (int i = 0; i < kKRing && issued[0] - i >= 0; ++i)
      drain_wait(x, x.bar(kKFull + (issued[0] - i) % kKRing), ((issued[0] - i) / kKRing) & 1, 13);
    for (int j = 0; j < 2; ++j)
      for (int i = 0; i < kVRing / 2 && issued[1 + j] - i >= 0; ++i) {
        const int v = 2 * (issued[1 + j] - i) + j;
        drain_wait(x, x.bar(kVFull + v % kVRing), (v / kVRing) & 1, 14);
      }
    if (issued[3] >= 0) drain_wait(x, x.bar(kQFull), issued[3] & 1, 15);
  }
  __syncwarp();
  fence_before_sync();
  cluster_sync();  // the pair's instructions and arrivals are done in both CTAs
  fence_after_sync();
  if (x.warp == 1) pair_dealloc(x.tbase, kTmemCols);
}

template <int BOX, Scale SCALE>
cudaError_t launch_variant(const PairMaps& maps, const DecodeParams& p, unsigned pairs, int* status,
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
  cfg.gridDim = dim3(2u * pairs);
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
cudaError_t launch_box(const PairMaps& maps, const DecodeParams& p, unsigned pairs, int* status, cudaStream_t stream) {
  if (p.kv_scales == nullptr) return launch_variant<BOX, Scale::kNone>(maps, p, pairs, status, stream);
  if (p.scale_group % kUni == 0) return launch_variant<BOX, Scale::kSixteen>(maps, p, pairs, status, stream);
  return launch_variant<BOX, Scale::kKey>(maps, p, pairs, status, stream);
}

}  // namespace

cudaError_t launch_decode_pair(const DecodeParams& p, int64_t q_rows, int64_t kv_rows, unsigned pairs, int* status,
                               cudaStream_t stream) {
  if (p.block_size % 16 != 0 || p.items == nullptr || p.worker_first == nullptr) return cudaErrorInvalidValue;
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
  return box == 64 ? launch_box<64>(maps, p, pairs, status, stream)
         : box == 32 ? launch_box<32>(maps, p, pairs, status, stream)
                     : launch_box<16>(maps, p, pairs, status, stream);
}

}  // namespace mla

// decode_vs.cu -- split-K paged MLA decode over an e4m3 cache with group
// scales, for row tiles of up to 128 query rows: two CTAs that split the value
// columns of a tile (sm_103a).
//
// The fp32 accumulator of 128 rows x 512 value columns fills a whole tensor
// memory, so a row tile takes two SMs. Here each CTA owns all 128 rows and 256
// of the value columns; both compute all scores and the same softmax. That
// doubles Q K^T, but nothing crosses between the SMs (probabilities would:
// distributed shared memory moves about 20 bytes a clock) and the epilogue is
// halved. Per chunk of 128 keys a CTA issues
//   S[rows, keys]  = Q K^T   M = 128 rows, N = 128 keys, K = 576: A = q from
//                            TMEM (512 latent dims) and shared memory (64 rope
//                            dims), B = the key rows of the rings, K-major:
//                            18 kind::f8f6f4 instructions of 64.5 cycles;
//   O[rows, 256]  += P V     for each half of 64 keys: M = 128 rows, N = 256
//                            columns, K = 64, P as two terms (hi in e4m3, lo in
//                            e5m2), V = the same key rows read MN-major: 8
//                            instructions a chunk of 128 cycles.
// That is 2180 tensor cycles a chunk, close to what the shared memory's 128
// bytes a clock allow for the operands, the copies in and P (284 KB, 2220
// cycles). Measured: 3100 to 3400 (52 x 16384 keys, 128 heads), bound by the
// chain S -> maxima -> weights -> P of a half-chunk (2600 cycles) and its
// hand-overs; at 1.7 GHz, as the SMs clock under this load, 188 us.
//
// The softmax works on half-chunks of 64 keys: one group of eight warps takes
// the even ones, another the odd ones, so that each has two of them in
// flight. A warp reads its 32 rows x 32 keys of S into registers and frees
// them at once: the next chunk's Q K^T runs while the weights are formed, and
// one buffer of S is enough. P has one for each half. (Groups on
// alternate whole chunks, with two buffers of S: 191 us against 183.)
//
// Rings: the two latent boxes of the own value columns stay until P V, the
// other two and the rope box only until Q K^T. They have rings of their own, of
// three, two and two chunks: what limits the loop is a box's lifetime (load,
// Q K^T, softmax, P V: about 8000 cycles for a value box), and in one ring of
// ten slots the short-lived boxes would wait behind the long-lived ones. The
// two CTAs of a tile read each key row once from memory between them: the later
// one finds it in L2. (Multicasting each box to both, from one read of L2, ties
// each slot to the slower CTA: 5930 cycles a chunk against 4730 without, when
// both had one ring.)
//
// Weights: with group scales the thread's scores become t = score + log2 s and
// the weights 2^(t - m) multiply the codes (KeyScale). They are formed as
// p = 2^(t - m_ref + 4) with a reference that moves only when a half-chunk's
// maximum exceeds it by more than 4.75 (O is then rescaled in TMEM), so p <=
// 2^8.75 fits e4m3; hi + lo carry 7 bits of it, and the rest of a weight down to
// 2^-21 of the row's largest (Rest: rows of which one key outweighs a long
// context).
//
// Warps: 0 loads, 1 issues Q K^T, 2 prepares the keys' scales (keys copied row by
// row: 0 and 2 share the copies), 3 issues P V, 4-19 softmax and epilogue (of either
// group: a TMEM lane quarter of the rows and half of the half-chunk's keys
// each). Every wait is bounded: a timeout records a code in the status word,
// stops the CTA's work, drains what was issued and exits.
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
constexpr int kKeys = 128;               // keys per chunk: N of Q K^T
constexpr int kHalf = 64;                // keys per half-chunk: of a TMA box, K of P V
constexpr int kSlot = kKeys * 128;       // ring slot: a 128-byte column box of a chunk (or of q)
constexpr int kRSlot = kKeys * 64;       // rope ring slot
constexpr int kKChunks = 2;              // ring of the other CTA's value columns (two boxes) and the
                                         // rope box: chunks
constexpr int kVChunks = 3;              // ring of the own value columns (two boxes): chunks
constexpr int kQStage = 2;               // q's latent boxes land in value slots 2..5 (chunks 1 and 2)
constexpr int kSoftWarps = 16;           // warps 4-19: two groups (even and odd half-chunks) of four
                                         // TMEM lane quarters x two key quarters
constexpr int kGroupWarps = 8;
constexpr int kPart = 32;                // keys of a softmax warp
constexpr int kUni = 16;                 // keys that share their scale where the groups are multiples of it
constexpr int kThreads = 32 * (4 + kSoftWarps);
constexpr int kPTile = kRows * kHalf;    // one term of P of a half-chunk
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;           // 256 columns
constexpr uint32_t kTmemS = 256;         // 128: S of a chunk
constexpr uint32_t kTmemQ = 384;         // 128: 512 latent dims, four to a column
constexpr uint64_t kDefaultWaitNs = 2000000000ull;
constexpr uint32_t kSleepNs = 20000;
// p = 2^(t - ref + kPBias); the reference moves when a half-chunk's maximum
// exceeds it by more than kMove, so that p <= 2^8.75 = 431 (e4m3 ends at 448)
// and a row's largest weight is at 2^4 or more.
constexpr float kPBias = 4.f;
constexpr float kMove = 4.75f;

enum : int {
  kFull = 0,                 // [kVChunks] chunk c loaded, at c % kVChunks: both kinds of boxes
  kKEmpty = kFull + kVChunks,   // [kKChunks] key and rope boxes released
  kVEmpty = kKEmpty + kKChunks,  // [kVChunks] value boxes released
  kQFull = kVEmpty + kVChunks,  // q staged
  kQTmem,                    // q copied to TMEM: the staging slots are free
  // of half-chunk g, at index g % 2:
  kSFull,                    // [2] S written and key scales ready
  kSFree = kSFull + 2,       // [2] S read
  kPFull = kSFree + 2,       // [2] P written
  kPFree = kPFull + 2,       // [2] P V complete: P may be replaced, O holds the half-chunk
  kX = kPFree + 2,           // [4][4] (at g % 4) the two warps of a row quarter have posted their maxima
  kScFree = kX + 16,         // [2] key scales of a chunk read
  kXL = kScFree + 2,         // [4] the four warps of a row quarter have posted their sums
  kDrain = kXL + 4,          // the Q K^T issuer's MMAs complete
  kDrainPV,
  kNumBars
};

// Shared memory: header, q's rope columns, P, the three rings.
constexpr int kOffBar = 0;
constexpr int kOffTslot = 512;
constexpr int kOffAbort = 516;
constexpr int kOffIssued = 576;           // [2][kVChunks] int: last chunk issued, by kind of boxes
constexpr int kOffMask = 640;             // [2][4] bits of existing keys of chunk c (at c % 2)
constexpr int kOffXMax = 768;             // [4][2][128] maxima of half-chunk g (at g % 4) by key quarter
constexpr int kOffScale = 4864;           // [2][mul, add, inv][128] of chunk c (at c % 2)
constexpr int kOffLsum = 7936;            // [4][128] row sums by group and key quarter
constexpr int kOffQR = 10240;             // 128 rows x 64 bytes, 64-byte swizzle
constexpr int kOffP = kOffQR + kRSlot;    // [g % 2][hi, lo] tiles of half-chunk g, 64-byte swizzle
constexpr int kOffRope = kOffP + 4 * kPTile;
constexpr int kOffKey = kOffRope + kKChunks * kRSlot;
constexpr int kOffVal = kOffKey + kKChunks * 2 * kSlot;
constexpr int kSmem = kOffVal + kVChunks * 2 * kSlot + 1024;  // + alignment slack
static_assert(kNumBars * 8 <= kOffTslot && kOffIssued + 8 * kVChunks <= kOffMask && kOffLsum + 2048 <= kOffQR,
              "header space");
static_assert(kSmem <= 232448, "shared memory budget");

// Box j of chunk c: 0, 1 of the other CTA's value columns, 2, 3 of the own, 4 the rope columns.
struct Box {
  int col, off;  // first column, shared memory
};
__device__ __forceinline__ Box box_of(int c, int j, int rank) {
  if (j < 2) return Box{128 * (2 * (rank ^ 1) + j), kOffKey + (2 * (c % kKChunks) + j) * kSlot};
  if (j < 4) return Box{128 * (2 * rank + j - 2), kOffVal + (2 * (c % kVChunks) + j - 2) * kSlot};
  return Box{kRank, kOffRope + c % kKChunks * kRSlot};
}

// Where the keys of a row tile are: in blocks of a multiple of 64 slots (TMA
// boxes), in blocks of any size, or in a list of slots (both copied row by row).
enum class Keys { kBoxes, kBlocks, kList };

struct VsMaps {
  CUtensorMap q;     // q as [T*H rows, 576] e4m3, box 128 bytes x 128 rows
  CUtensorMap qr;    // the same, box 64 bytes (the rope columns)
  CUtensorMap kv;    // cache as [NB*BS rows, 576], box 128 bytes x 64 rows (Keys::kBoxes)
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
  int seg, seg_start, seg_end, n_chunks, n_half;  // chunks of 128 keys, half-chunks of 64
  int pslot;  // partial slot of a balanced piece, -1: write out/lse
  bool fin;
  __device__ uint32_t bar(int i) const { return bar0 + 8u * i; }
};

// Largest of three (one instruction; NaN is passed over).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 operations in one instruction.
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

__device__ __forceinline__ void report(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// Bounded wait on a barrier phase, sleeping; false on timeout (recorded) or abort.
__device__ bool wait_phase(const Ctx& x, uint32_t bar, uint32_t parity, int code) {
  const bool brief = x.limit_ns < kSleepNs;  // (a sleep may last longer than the limit: poll)
  if (mbar_test_wait(bar, parity)) return true;
  // one sleep before the clock is read for the first time: nearly every wait
  // ends in it, and reading the global timer takes longer than most waits
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

// Cache slot of key position pos (-1 past the segment; negative for an unused list
// entry and where the table has no block).
template <bool LIST>
__device__ __forceinline__ int key_slot(const Ctx& x, const DecodeParams& p, const int32_t* bt_row, int pos) {
  if (pos >= x.seg_end) return -1;
  if constexpr (LIST) return p.slots[x.list_base + pos];
  const int blk = pos / p.block_size;
  return bt_row[blk] * p.block_size + (pos - blk * p.block_size);
}

// ------------------------------------------------------------------ producers
// The slots of a chunk's value boxes (or its others) may be filled: their last
// use is released and, where q is staged there, q has left. Uniform in the warp.
template <bool VALUES>
__device__ __forceinline__ bool slots_ready(const Ctx& x, int c) {
  constexpr int kRing = VALUES ? kVChunks : kKChunks;
  if (c >= kRing) return warp_wait(x, x.bar((VALUES ? kVEmpty : kKEmpty) + c % kRing), (c / kRing - 1) & 1, 11);
  return !VALUES || c == 0 || warp_wait(x, x.bar(kQTmem), 0, 10);
}
// One arrival for either kind, with the bytes to come, on the chunk's barrier.
template <bool VALUES>
__device__ __forceinline__ uint32_t announce(const Ctx& x, int c, uint32_t bytes) {
  const uint32_t full = x.bar(kFull + c % kVChunks);
  if (x.lane == 0) {
    mbar_arrive_expect_tx(full, bytes);
    reinterpret_cast<volatile int*>(x.smem + kOffIssued)[(VALUES ? kVChunks : 0) + c % kVChunks] = c;
  }
  __syncwarp();
  return full;
}

// Dense: warp 0 loads a chunk's boxes, first those that wait for Q K^T alone,
// then the value boxes. Each is two 64-row TMA boxes from their blocks, one by
// each of two lanes; the boxes of one kind go out together (a lane issuing
// them in turn takes about 350 cycles each, which alone held the loop at 4240
// cycles a chunk).
template <bool VALUES>
__device__ __forceinline__ bool load_boxes(const Ctx& x, const VsMaps& maps, int c, int row0, int row1) {
  constexpr int kCount = VALUES ? 2 : 3;
  const int lane = x.lane;
  const bool two = 2 * c + 1 < x.n_half;
  if (!slots_ready<VALUES>(x, c)) return false;
  const uint32_t full = announce<VALUES>(x, c, (2 * kSlot + (VALUES ? 0 : kRSlot)) >> (two ? 0 : 1));
  if (lane < 2 * kCount && ((lane & 1) == 0 || two)) {
    const int i = lane >> 1;
    const bool rope = i == 2;
    const Box b = box_of(c, VALUES ? 2 + i : rope ? 4 : i, x.rank);
    tma_load_2d(smem_u32(x.smem + b.off + (lane & 1) * ((rope ? kRSlot : kSlot) / 2)), rope ? &maps.kvr : &maps.kv,
                b.col, (lane & 1) != 0 ? row1 : row0, full);
  }
  __syncwarp();
  return true;
}

// The rows of a chunk's keys into its boxes, in their swizzles, by
// 16-byte asynchronous copies: an instruction takes 128 bytes of four rows (of
// the rope columns: 64 of eight). v[k] of lane l is the cache slot of key
// 32 k + l; a key without one is filled with zeros. (TMA's row gathers take
// about 13 cycles a row of 128 bytes: 8500 cycles a chunk.)
enum : int { kOther = 0, kOwn = 2, kRope = 4 };  // first box (box_of) of a share
template <int FIRST>
__device__ __forceinline__ void copy_rows(const Ctx& x, const DecodeParams& p, int c, const int (&v)[4]) {
  constexpr int kLanes = FIRST == kRope ? 4 : 8;  // of a row
  constexpr int kStep = 32 / kLanes;              // keys an instruction
  const int key = x.lane / kLanes, piece = x.lane % kLanes;
  const Box b = box_of(c, FIRST, x.rank);
  const uint8_t* from = static_cast<const uint8_t*>(p.kv) + b.col + 16 * piece;
  const uint32_t to = smem_u32(x.smem + b.off) + 16 * kLanes * key +
                      ((FIRST == kRope ? piece ^ ((key >> 1) & 3) : piece ^ key) << 4);
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int j = 0; j < kLanes; ++j) {
      const int s = __shfl_sync(0xffffffffu, v[k], kStep * j + key);
      const uint8_t* row = from + static_cast<int64_t>(max(s, 0)) * kHeadDim;
      const uint32_t n = s >= 0 ? 16u : 0u;
      if constexpr (FIRST == kRope) {
        cp_async_16(to + 512 * (kLanes * k + j), row, n);
      } else {  // (odd steps have bit 2 of the key set)
        const uint32_t at = (to ^ ((j & 1) << 6)) + 512 * (kLanes * k + j);
        cp_async_16(at, row, n);
        cp_async_16(at + kSlot, row + 128, n);
      }
    }
}

// Cache rows of the 64-key halves of a dense request's chunks: looked up by
// the whole warp, 16 chunks at a time and a window ahead. A half past the end or
// without a block has row -64, whose box is filled with zeros.
struct RowWindow {
  int cur, nxt;
  __device__ __forceinline__ void load(const Ctx& x, const DecodeParams& p, const int32_t* bt_row, int w0, int& v) {
    const int s =
        key_slot<false>(x, p, bt_row, x.seg_start + (w0 + (x.lane >> 1)) * kKeys + (x.lane & 1) * kHalf);
    v = s < 0 ? -kHalf : s;
  }
  __device__ __forceinline__ void start(const Ctx& x, const DecodeParams& p, const int32_t* bt_row) {
    load(x, p, bt_row, 0, cur);
    load(x, p, bt_row, 16, nxt);
  }
  // moves on to the window of chunk g (called for every chunk in turn)
  __device__ __forceinline__ void at(const Ctx& x, const DecodeParams& p, const int32_t* bt_row, int g) {
    if (g > 0 && (g & 15) == 0) {
      cur = nxt;
      load(x, p, bt_row, g + 16, nxt);
    }
  }
  __device__ __forceinline__ int row(int g, int half) const {
    return __shfl_sync(0xffffffffu, cur, 2 * (g & 15) + half);
  }
};

__device__ void produce_dense(const Ctx& x, const VsMaps& maps, const DecodeParams& p) {
  if (x.lane == 0) {
    tma_prefetch_desc(&maps.kv);
    tma_prefetch_desc(&maps.kvr);
  }
  const int32_t* bt_row = p.block_table + static_cast<int64_t>(x.unit) * p.bt_stride;
  RowWindow w;
  w.start(x, p, bt_row);
  for (int g = 0; g < x.n_chunks; ++g) {
    w.at(x, p, bt_row, g);
    const int row0 = w.row(g, 0), row1 = w.row(g, 1);
    if (!load_boxes<false>(x, maps, g, row0, row1) || !load_boxes<true>(x, maps, g, row0, row1)) break;
  }
  __syncwarp();
}

// The scale of slot s (s >= 0): its group by a multiplication (scale_magic).
__device__ __forceinline__ float scale_of_slot(const DecodeParams& p, int s) {
  const uint32_t g = p.scale_magic != 0 ? __umulhi(static_cast<uint32_t>(s), p.scale_magic) >> p.scale_shift
                                        : static_cast<uint32_t>(s) >> p.scale_shift;
  return __ldg(p.kv_scales + g);
}

// Posts the key scales of chunk c (part i of 32 keys: lane's key 32 i + lane;
// UNI: lane i < 8 has the scale of the 16 keys from 16 i) and the bits of the keys that exist,
// once the softmax has read those two chunks back. The half-chunks' S barriers
// count the post as well as Q K^T.
template <bool UNI>
__device__ __forceinline__ bool post_scales(const Ctx& x, const DecodeParams& p, int c, const float (&sc)[4],
                                            uint32_t bits) {
  const int lane = x.lane;
  if (c >= 2 && !warp_wait(x, x.bar(kScFree + (c & 1)), ((c >> 1) - 1) & 1, 27)) return false;
  float* ks = reinterpret_cast<float*>(x.smem + kOffScale) + (c & 1) * 3 * kKeys;
  if (lane < 4) reinterpret_cast<uint32_t*>(x.smem + kOffMask)[(c & 1) * 4 + lane] = bits;
#pragma unroll
  for (int i = 0; i < (UNI ? 1 : 4); ++i) {
    const KeyScale k = key_scale(sc[i], p.score_scale_log2);
    const int at = UNI ? kUni * lane : 32 * i + lane;
    if (!UNI || lane < kKeys / kUni) {
      ks[at] = k.mul;
      ks[kKeys + at] = k.add;
      ks[2 * kKeys + at] = k.inv;
    }
  }
  __syncwarp();
  const int nh = min(2, x.n_half - 2 * c);
  for (int h = 0; h < nh; ++h) {
    const uint32_t bar = x.bar(kSFull + h);
    if (c >= 1 && !warp_wait(x, bar, (c - 1) & 1, 28)) return false;  // S of the chunk before
    if (lane == 0) mbar_arrive(bar);
  }
  return true;
}

// Warp 2, dense: the scales, read one chunk ahead of the one posted.
template <bool UNI>
__device__ void scales_dense(const Ctx& x, const DecodeParams& p) {
  const int lane = x.lane;
  const int32_t* bt_row = p.block_table + static_cast<int64_t>(x.unit) * p.bt_stride;
  RowWindow w;
  w.start(x, p, bt_row);
  float sc[4];
  uint32_t bits = 0u;  // lane i < 4: the keys of part i that exist
  auto read = [&](int g) {  // 1 for keys that do not exist
    w.at(x, p, bt_row, g);
    const int row0 = w.row(g, 0), row1 = w.row(g, 1);
    const int n = x.seg_end - (x.seg_start + g * kKeys);
#pragma unroll
    for (int i = 0; i < (UNI ? 1 : 4); ++i) {
      const int j = UNI ? kUni * lane : 32 * i + lane;
      const int row = j < kHalf ? row0 : row1;
      sc[i] = j < n && j < kKeys && row >= 0 ? scale_of_slot(p, row + (j & (kHalf - 1))) : 1.f;
    }
    const int left = (lane < 2 ? row0 : row1) >= 0 ? n - 32 * lane : 0;
    bits = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
  };
  if (x.n_chunks > 0) read(0);
  for (int g = 0; g < x.n_chunks; ++g) {
    if (!post_scales<UNI>(x, p, g, sc, bits)) break;
    if (g + 1 < x.n_chunks) read(g + 1);
  }
  __syncwarp();
}

// Keys copied row by row: warp 0 (VALUES) copies the own value boxes and the
// rope columns, warp 2 the other boxes, and prepares the scales. The slots of a lane's keys
// are read a chunk ahead. A chunk is posted when its copies, issued an
// iteration before, have landed.
template <bool LIST, bool VALUES>
__device__ void produce_rows(const Ctx& x, const DecodeParams& p) {
  const int lane = x.lane;
  const int32_t* bt_row = LIST ? nullptr : p.block_table + static_cast<int64_t>(x.unit) * p.bt_stride;
  int slot[4], next[4];
  float sc[4];
  auto slots_of = [&](int g, int (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = g < x.n_chunks ? key_slot<LIST>(x, p, bt_row, x.seg_start + g * kKeys + 32 * i + lane) : -1;
  };
  auto scales_of = [&](const int (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = v[i] >= 0 ? scale_of_slot(p, v[i]) : 1.f;
  };
  slots_of(0, next);
  for (int g = 0; g <= x.n_chunks; ++g) {
    if (g > 0) {  // the copies of g - 1 are complete: make them visible to the MMAs
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(x.bar(kFull + (g - 1) % kVChunks));
    }
    if (g == x.n_chunks) break;
    // (after the fence, which waits for loads)
#pragma unroll
    for (int i = 0; i < 4; ++i) slot[i] = next[i];
    if constexpr (!VALUES) scales_of(slot);
    slots_of(g + 1, next);
    if (!slots_ready<VALUES>(x, g) || (VALUES && !slots_ready<false>(x, g))) break;
    copy_rows<VALUES ? kOwn : kOther>(x, p, g, slot);
    if constexpr (VALUES) copy_rows<kRope>(x, p, g, slot);
    cp_async_commit();
    if constexpr (!VALUES) {
      uint32_t bits = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = __ballot_sync(0xffffffffu, slot[i] >= 0);
        if (lane == i) bits = b;
      }
      if (!post_scales<false>(x, p, g, sc, bits)) break;
    }
  }
  cp_async_wait<0>();  // also where a wait gave up: no copy outlives the CTA
  __syncwarp();
}

// ------------------------------------------------------------------ MMA issue
// The issuing warps stay together: addresses and descriptors are computed
// uniformly and one elected lane issues. (A lane on its own, with the values
// in its vector registers, took about 165 cycles an instruction between the
// softmax warps of its scheduler, more than twice its 64 tensor cycles.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Four steps of 32 columns of a 128-byte column box: D (+)= A[tmem] B[smem].
__device__ __forceinline__ void mma_box(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b32 l, t;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n"
      " mov.b64 b, {%2, %3};\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], b, %4, p;\n"
      " add.u32 l, %2, 2;\n add.u32 t, %1, 8;\n mov.b64 b, {l, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [t], b, %4, 1;\n"
      " add.u32 l, %2, 4;\n add.u32 t, %1, 16;\n mov.b64 b, {l, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [t], b, %4, 1;\n"
      " add.u32 l, %2, 6;\n add.u32 t, %1, 24;\n mov.b64 b, {l, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [t], b, %4, 1;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Position in a ring of N chunks, and the phase parity of its slots.
template <int N>
struct RingPos {
  int at = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

__device__ void qk_issue(const Ctx& x, const VsMaps& maps) {
  if (x.n_chunks == 0) return;
  constexpr uint32_t kId = instr_desc(kRows, kKeys, 0, 0, false, false);
  const uint32_t base = smem_u32(x.smem);
  const uint64_t k_desc = smem_desc_sw128(base, 16, 1024);
  const uint64_t r_desc = smem_desc_sw64(base + kOffRope, 512);
  const uint64_t q_desc = smem_desc_sw64(base + kOffQR, 512);
  const uint32_t k_lo = static_cast<uint32_t>(k_desc), k_hi = static_cast<uint32_t>(k_desc >> 32);
  const bool one = elect_one();
  if (one) {
    tma_prefetch_desc(&maps.q);
    mbar_arrive_expect_tx(x.bar(kQFull), 4 * kSlot + kRSlot);
    const int qrow = x.tok0 * x.H + x.row0;
    for (int j = 0; j < 4; ++j)
      tma_load_2d(base + kOffVal + (kQStage + j) * kSlot, &maps.q, 128 * j, qrow, x.bar(kQFull));
    tma_load_2d(base + kOffQR, &maps.qr, kRank, qrow, x.bar(kQFull));
  }
  __syncwarp();
  bool ok = warp_wait(x, x.bar(kQFull), 0, 20) && warp_wait(x, x.bar(kQTmem), 0, 21);
  const uint32_t a_key = x.tbase + kTmemQ + 64u * (x.rank ^ 1), a_val = x.tbase + kTmemQ + 64u * x.rank;
  RingPos<kKChunks> kr;
  RingPos<kVChunks> vr;
  const uint32_t d = x.tbase + kTmemS;
  for (int c = 0; c < x.n_chunks; ++c) {
    // (a last chunk of one half multiplies whatever the rows of the other hold:
    // nobody reads those scores)
    const bool two = 2 * c + 1 < x.n_half;
    ok = ok && warp_wait(x, x.bar(kFull + vr.at), vr.phase, 23);
    ok = ok && (c < 1 || (warp_wait(x, x.bar(kSFree), (c - 1) & 1, 22) &&
                          warp_wait(x, x.bar(kSFree + 1), (c - 1) & 1, 29)));
    if (!ok) break;
    fence_after_sync();
    const uint32_t lo_k = k_lo + ((kOffKey + kr.at * 2 * kSlot) >> 4);
    const uint32_t lo_v = k_lo + ((kOffVal + vr.at * 2 * kSlot) >> 4);
    const uint64_t rd = r_desc + static_cast<uint64_t>((kr.at * kRSlot) >> 4);
    if (one) {
      mma_box(d, a_key, lo_k, k_hi, kId, 0u);
      mma_box(d, a_key + 32u, lo_k + (kSlot >> 4), k_hi, kId, 1u);
      mma_box(d, a_val, lo_v, k_hi, kId, 1u);
      mma_box(d, a_val + 32u, lo_v + (kSlot >> 4), k_hi, kId, 1u);
      mma_ss_f8(d, q_desc, rd, kId, 1u);
      mma_ss_f8(d, q_desc + 2, rd + 2, kId, 1u);
      mma_commit(x.bar(kSFull));
      if (two) mma_commit(x.bar(kSFull + 1));
      mma_commit(x.bar(kKEmpty + kr.at));  // the key and rope boxes' only reads
    }
    __syncwarp();
    kr.next();
    vr.next();
  }
  if (one) {
    mma_commit(x.bar(kDrain));
    drain_wait(x, x.bar(kDrain), 0, 25);
  }
  __syncwarp();
}

// The own value rows of keys [first, end) of half-chunk g, without NaNs.
__device__ __forceinline__ void drop_nans(const Ctx& x, int g, int first, int end) {
  uint8_t* box = x.smem + box_of(g >> 1, 2, x.rank).off + (g & 1) * kHalf * 128;
#pragma unroll 1
  for (int i = first * 16 + x.lane; i < end * 16; i += 32) {
    uint4* at = reinterpret_cast<uint4*>(box + ((i >> 3) & 1) * kSlot + (i >> 4) * 128 + (i & 7) * 16);
    const uint4 v = *at;
    *at = make_uint4(e4m3x4_without_nan(v.x), e4m3x4_without_nan(v.y), e4m3x4_without_nan(v.z), e4m3x4_without_nan(v.w));
  }
  fence_proxy_async_smem();
  __syncwarp();
}

__device__ void pv_issue(const Ctx& x, const DecodeParams& p) {
  if (x.n_chunks == 0) return;
  constexpr uint32_t kIdHi = instr_desc(kRows, 256, 0, 0, false, true);
  constexpr uint32_t kIdLo = instr_desc(kRows, 256, 1, 0, false, true);
  const uint64_t v_desc = smem_desc_sw128(smem_u32(x.smem + kOffVal), kSlot, 1024);  // MN-major, two boxes
  const uint64_t p_desc = smem_desc_sw64(smem_u32(x.smem + kOffP), 512);
  const uint32_t d = x.tbase + kTmemO;
  const bool one = elect_one();
  RingPos<kVChunks> vr;
  auto step = [&](int g) {
    const int h = g & 1;
    const bool last = h == 1 || g + 1 == x.n_half;
    // P written; the softmax waited for S, whose Q K^T waited for these boxes
    if (!warp_wait(x, x.bar(kPFull + h), (g >> 1) & 1, 24)) return false;
    fence_after_sync();
    const uint64_t vb = v_desc + static_cast<uint64_t>((vr.at * 2 * kSlot + h * kHalf * 128) >> 4);
    const uint64_t pb = p_desc + static_cast<uint64_t>((h * 2 * kPTile) >> 4);
    if (one) {
#pragma unroll
      for (int ks = 0; ks < kHalf / 32; ++ks) {
        const uint64_t av = pb + static_cast<uint64_t>((ks * 32) >> 4);
        const uint64_t bv = vb + static_cast<uint64_t>((ks * 32 * 128) >> 4);
        mma_ss_f8(d, av, bv, kIdHi, (g | ks) != 0 ? 1u : 0u);
        mma_ss_f8(d, av + static_cast<uint64_t>(kPTile >> 4), bv, kIdLo, 1u);
      }
      if (last) mma_commit(x.bar(kVEmpty + vr.at));
      mma_commit(x.bar(kPFree + h));
    }
    __syncwarp();
    if (last) vr.next();
    return true;
  };
  // keys before all_see are seen by every row of the tile; of those from it on a
  // NaN must not reach the rows that do not see them through p = 0. (A loop of
  // their own, from lengths read again: a test in the other loop cost 2 % of
  // every call, the values kept in registers spilled the softmax's.)
  const int qlen = p.qo_indptr != nullptr ? p.qo_indptr[x.unit + 1] - p.qo_indptr[x.unit] : 1;
  const int all_see = qlen > 1 ? p.seq_lens[x.unit] - qlen + x.row0 / p.num_heads + 1 - x.seg_start : 0;
  const int tail = qlen > 1 ? min(max(all_see, 0) / kHalf, x.n_half) : x.n_half;
  bool ok = true;
  for (int g = 0; g < tail && ok; ++g) ok = step(g);
#pragma unroll 1
  for (int g = tail; g < x.n_half && ok; ++g) {
    ok = warp_wait(x, x.bar(kPFull + (g & 1)), (g >> 1) & 1, 24) &&
         warp_wait(x, x.bar(kFull + vr.at), vr.phase, 39);  // (the box has landed; this shows its writes)
    if (!ok) break;
    drop_nans(x, g, max(all_see - g * kHalf, 0), min(x.seg_end - x.seg_start - g * kHalf, kHalf));
    ok = step(g);
  }
  if (one) {
    mma_commit(x.bar(kDrainPV));
    drain_wait(x, x.bar(kDrainPV), 0, 26);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax + epilogue
template <Keys KEYS, bool UNI>
__device__ void softmax_rows(const Ctx& x, const VsMaps& maps, const DecodeParams& p) {
  const int lane = x.lane;
  const int sw = x.warp - 4;
  const int q4 = x.warp & 3;               // TMEM lane quarter of this warp
  const int h = sw >> 3;                   // half-chunks g with g % 2 == h: half of its chunk, and buffer
  const int kh = (sw >> 2) & 1;            // its 32 keys of a half-chunk
  const int cq = sw >> 2;                  // its box of q, and quarter of the CTA's value columns at the end
  const int r = q4 * 32 + lane;            // row within the tile
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const int H = x.H;
  const int rho = x.row0 + r;
  const bool row_ok = rho < x.rows_total;
  const int vis = !row_ok ? 0 : (KEYS == Keys::kList ? INT_MAX : x.part_len - x.qlen + rho / H + 1);
  const int n = x.n_half;
  bool ok = true;

  // this row of q, staged in the value ring, into TMEM (one of the four
  // latent boxes each)
  if (n > 0) {
    ok = warp_wait(x, x.bar(kQFull), 0, 30);
    if (ok) {
      const uint8_t* src = x.smem + kOffVal + (kQStage + cq) * kSlot + r * 128;
      uint32_t v[32];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint4 t = *reinterpret_cast<const uint4*>(src + ((q ^ (r & 7)) << 4));
        v[4 * q] = t.x;
        v[4 * q + 1] = t.y;
        v[4 * q + 2] = t.z;
        v[4 * q + 3] = t.w;
      }
      tmem_st_32x32b_x32(x.tbase + lane_off + kTmemQ + 32 * cq, v);
      tmem_st_wait();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(x.bar(kQTmem));
    }
  }

  float* xmax = reinterpret_cast<float*>(x.smem + kOffXMax) + r;
  // the warp's keys in P: two 16-byte chunks of the row's 64 bytes of either
  // tile, 64-byte swizzle
  uint8_t* prow = x.smem + kOffP + h * 2 * kPTile + r * 64;
  const int c0 = ((2 * kh) ^ ((r >> 1) & 3)) << 4, c1 = ((2 * kh + 1) ^ ((r >> 1) & 3)) << 4;
  const uint32_t ts = x.tbase + lane_off + kTmemS + kHalf * h + kPart * kh;

  // Every thread follows its row's reference through the maxima of all
  // half-chunks: it moves to one that exceeds it by more than kMove. Returns
  // the factor of what was formed before.
  float ref = -INFINITY, l = 0.f;
  auto follow = [&](float mx) {
    if (!(mx > ref + kMove)) return 1.f;  // (moves also when a row's first visible key arrives)
    const float a = ref == -INFINITY ? 1.f : fast_exp2(ref - mx);
    ref = mx;
    l *= a;
    return a;
  };
  // the maximum of half-chunk g, which two warps of the other group posted. A
  // group looks at it before it posts its own of g + 1, which the other waits
  // for before it posts that of g + 4: neither the barrier's phase nor the four
  // buffers are passed over.
  auto follow_other = [&](int g) {
    if (!warp_wait(x, x.bar(kX + 4 * (g & 3) + q4), (g >> 2) & 1, 33)) return false;
    const float* xm = xmax + (g & 3) * 2 * kRows;
    follow(fmaxf(xm[0], xm[kRows]));
    return true;
  };
  for (int g = h; g < n && ok; g += 2) {
    const int ph = (g >> 1) & 1;
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
    if (lane == 0) mbar_arrive(x.bar(kSFree + h));  // the next chunk's Q K^T may overwrite it
    const int sst = (g >> 1) & 1;                   // stage of the chunk's scales
    const float* ks = reinterpret_cast<const float*>(x.smem + kOffScale) + sst * 3 * kKeys + kHalf * h + kPart * kh;
    const uint32_t kmask = reinterpret_cast<const uint32_t*>(x.smem + kOffMask)[4 * sst + 2 * h + kh];
    if constexpr (!UNI) {
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
    const int lim = min(vis, x.seg_end) - (x.seg_start + g * kHalf + kPart * kh);
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
    }
    const float mine = fmaxf(m[0], m[1]);
    // the row's maximum over both key quarters; the previous half-chunk's before it
    ok = g == 0 || follow_other(g - 1);
    if (!ok) break;
    float* xm = xmax + (g & 3) * 2 * kRows;
    xm[kh * kRows] = mine;
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kX + 4 * (g & 3) + q4));
    ok = warp_wait(x, x.bar(kX + 4 * (g & 3) + q4), (g >> 2) & 1, 32);
    if (!ok) break;
    const float alpha = follow(fmaxf(mine, xm[(kh ^ 1) * kRows]));
    // p as hi + lo terms, 16 keys to a 16-byte chunk of each tile
    const float base = ref == -INFINITY ? 0.f : ref - kPBias;
    float psum = 0.f;
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mu = UNI ? ks[kUni * i] : 1.f, sh = UNI ? ks[kKeys + kUni * i] - base : -base;
      const float2 mul2 = make_float2(mu, mu), shift2 = make_float2(sh, sh);
      float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int j = 4 * i; j < 4 * i + 4; ++j) {
        const int e = 4 * j;
        float2 a = make_float2(s[e], s[e + 1]), b = make_float2(s[e + 2], s[e + 3]);
        a = UNI ? fma2(a, mul2, shift2) : add2(a, shift2);
        b = UNI ? fma2(b, mul2, shift2) : add2(b, shift2);
        a = make_float2(fast_exp2(a.x), fast_exp2(a.y));
        b = make_float2(fast_exp2(b.x), fast_exp2(b.y));
        if constexpr (UNI) {
          ps[0] = add2(ps[0], a);
          ps[1] = add2(ps[1], b);
        } else {
          const float4 iv = *reinterpret_cast<const float4*>(ks + 2 * kKeys + e);
          ps[0] = fma2(a, make_float2(iv.x, iv.y), ps[0]);
          ps[1] = fma2(b, make_float2(iv.z, iv.w), ps[1]);
        }
        p_terms4(a.x, a.y, b.x, b.y, hi[j], lo[j]);
      }
      const float sum = (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y);
      psum = UNI ? fmaf(sum, ks[2 * kKeys + kUni * i], psum) : psum + sum;
    }
    l += psum;
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kScFree + sst));
    // P V two half-chunks back has read this buffer of P
    ok = g < 2 || warp_wait(x, x.bar(kPFree + h), ph ^ 1, 37);
    if (!ok) break;
    *reinterpret_cast<uint4*>(prow + c0) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(prow + c1) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
    *reinterpret_cast<uint4*>(prow + kPTile + c0) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(prow + kPTile + c1) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
    if (__any_sync(0xffffffffu, alpha != 1.f)) {
      // some rows moved their reference: once O is complete up to the previous
      // half-chunk, this warp rescales its rows of its half of the value
      // columns. (This barrier's phase before, P V of g - 3, completed with that
      // of g - 2, as P V is issued in order: the parity cannot be taken for it.)
      ok = warp_wait(x, x.bar(kPFree + (h ^ 1)), ((g - 1) >> 1) & 1, 38);
      if (!ok) break;
      fence_after_sync();
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        const uint32_t ta = x.tbase + lane_off + kTmemO + 128 * kh + 64 * c;
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
    // value rows of keys that do not exist (stale ring contents, cache rows past
    // the sequence, unused list entries) must not reach O through p = 0: they
    // are zeroed, a quarter by each warp
    if (KEYS == Keys::kBoxes && kmask != 0xffffffffu) {
      uint8_t* box = x.smem + box_of(g >> 1, 2, x.rank).off + ((lane >> 3) & 1) * kSlot +
                     (kHalf * h + kPart * kh) * 128 + (lane & 7) * 16;
      for (int j = q4 + 4 * (lane >> 4); j < kPart; j += 8)
        if (!((kmask >> j) & 1u)) *reinterpret_cast<uint4*>(box + j * 128) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kPFull + h));
  }

  // ---------------------------------------------------------------- epilogue
  if (ok && n > 0 && ((n - 1) & 1) != h) ok = follow_other(n - 1);  // the last one was the other group's
  float* lsum = reinterpret_cast<float*>(x.smem + kOffLsum) + r;
  if (ok) {
    lsum[cq * kRows] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kXL + q4));
    ok = warp_wait(x, x.bar(kXL + q4), 0, 34);
  }
  // O is complete with the last half-chunk (the phase before of its barrier, P V
  // of n - 3, was waited for by its group before it posted its sum)
  if (ok && n > 0) {
    ok = warp_wait(x, x.bar(kPFree + ((n - 1) & 1)), ((n - 1) >> 1) & 1, 35);
    fence_after_sync();
  }
  if (!ok) return;
  float mult = 0.f;
  if (row_ok) {
    const float L = (lsum[0] + lsum[kRows]) + (lsum[2 * kRows] + lsum[3 * kRows]);
    const float base = ref == -INFINITY ? 0.f : ref - kPBias;  // the reference of O and the sum
    const int head = rho % H;
    const int64_t th = static_cast<int64_t>(x.tok0 + rho / H) * H + head;
    const bool writes = x.rank == 0 && cq == 0;
    if (x.fin) {
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
        const int64_t ts = x.pslot >= 0 ? static_cast<int64_t>(x.pslot) * p.slot_rows + r : th * p.num_segments + x.seg;
        // (any reference of the partial serves the merge)
        const float2 part = partial_sums(L > 0.f ? base : -INFINITY, L);
        p.segm_max[ts] = part.x;
        p.segm_expsum[ts] = part.y;
      }
    }
  }
  // Each warp scales its 32 rows x 64 columns and stages them, 128 bytes of
  // each row at a time, in the 128-byte swizzle, in the rings (which hold no
  // more boxes in use). When all 32 rows are valid one TMA tensor store writes
  // each staged tile; otherwise every store instruction covers four 128-byte
  // row pieces. (TMEM loads are warp-collective.)
  const int col0 = 256 * x.rank + 64 * cq;
  const int wr = x.row0 + 32 * q4;          // the warp's first row within the unit
  if (wr >= x.rows_total) return;
  const bool whole = wr + 32 <= x.rows_total;
  const int z0 = x.fin || x.pslot < 0 ? x.tok0 * H + wr : x.pslot * p.slot_rows + 32 * q4;
  const int y0 = x.fin || x.pslot >= 0 ? 0 : x.seg;
  const CUtensorMap* map = x.fin ? &maps.out : &maps.part;
  const int qc = lane & 7;                  // 16-byte piece of a 128-byte row piece
  auto store = [&](const uint32_t (&w)[32], int col, int tile) {
    uint8_t* buf = x.smem + kOffKey + sw * 8192 + tile * 4096;
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
    }
  };
  if (x.fin) {
    uint32_t w[32];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t o[32];
      if (x.n_chunks > 0) {
        tmem_ld_32x32b_x32(x.tbase + lane_off + kTmemO + 64 * cq + 32 * c, o);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0u;
      }
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
      if (x.n_chunks > 0) {
        tmem_ld_32x32b_x32(x.tbase + lane_off + kTmemO + 64 * cq + 32 * c, o);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0u;
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * mult);
      store(o, col0 + 32 * c, c);
    }
  }
  if (lane == 0) bulk_wait_all();  // tiles read and written before the CTA exits
  __syncwarp();
}

template <Keys KEYS, bool UNI>
__global__ void __launch_bounds__(kThreads, 1)
    decode_vs_kernel(const __grid_constant__ VsMaps maps, const DecodeParams p, int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctx x;
  x.smem = smem;
  x.status = status;
  x.limit_ns = p.wait_ns != 0 ? p.wait_ns : kDefaultWaitNs;
  x.tid = threadIdx.x;
  x.warp = __shfl_sync(0xffffffffu, x.tid >> 5, 0);  // uniform, for the compiler too
  x.lane = x.tid & 31;
  x.rank = static_cast<int>(blockIdx.x & 1);
  int tile, item_begin = 0, item_end = 0;
  x.pslot = -1;
  if (p.items != nullptr) {
    // balanced schedule: both CTAs of a tile read the same item, once the grid
    // that wrote the list has completed; the merge may launch once every CTA
    // has started
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
  if constexpr (KEYS == Keys::kList) {
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
  if (x.row0 >= x.rows_total) return;
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
  x.n_half = x.seg_end > x.seg_start ? cdiv(x.seg_end - x.seg_start, kHalf) : 0;
  x.n_chunks = cdiv(x.n_half, 2);

  x.bar0 = smem_u32(smem + kOffBar);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + kOffTslot);
  x.abort = reinterpret_cast<volatile int*>(smem + kOffAbort);
  if (x.tid == 0) {
    *x.abort = 0;
    for (int i = 0; i < kVChunks; ++i) {
      mbar_init(x.bar(kFull + i), 2);
      mbar_init(x.bar(kVEmpty + i), 1);
    }
    for (int i = 0; i < kKChunks; ++i) mbar_init(x.bar(kKEmpty + i), 1);
    mbar_init(x.bar(kQFull), 1);
    mbar_init(x.bar(kQTmem), kSoftWarps);
    for (int b = 0; b < 2; ++b) {
      mbar_init(x.bar(kSFull + b), 2);  // Q K^T and the key scales
      mbar_init(x.bar(kSFree + b), kGroupWarps);
      mbar_init(x.bar(kPFull + b), kGroupWarps);
      mbar_init(x.bar(kPFree + b), 1);
      mbar_init(x.bar(kScFree + b), 2 * kGroupWarps);
    }
    for (int q = 0; q < 16; ++q) mbar_init(x.bar(kX + q), 2);
    for (int q = 0; q < 4; ++q) mbar_init(x.bar(kXL + q), 4);
    mbar_init(x.bar(kDrain), 1);
    mbar_init(x.bar(kDrainPV), 1);
    fence_barrier_init();
  }
  if (x.tid < 2 * kVChunks) reinterpret_cast<int*>(smem + kOffIssued)[x.tid] = -1;
  if (x.warp == 1) {
    tmem_alloc(smem_u32(tslot), kTmemCols);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  x.tbase = *tslot;

  if (x.warp >= 4) {
    softmax_rows<KEYS, UNI>(x, maps, p);
  } else if (x.warp == 1) {
    qk_issue(x, maps);
  } else if (x.warp == 3) {
    pv_issue(x, p);
  } else if (x.warp == 0) {
    if constexpr (KEYS == Keys::kBoxes)
      produce_dense(x, maps, p);
    else
      produce_rows<KEYS == Keys::kList, true>(x, p);
  } else {
    if constexpr (KEYS == Keys::kBoxes)
      scales_dense<UNI>(x, p);
    else
      produce_rows<KEYS == Keys::kList, false>(x, p);
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (x.warp == 1) tmem_dealloc(x.tbase, kTmemCols);
  // every load must have landed before the CTA exits: of each chunk's barrier,
  // the last chunk issued (all were consumed unless a wait gave up; where it
  // did between a chunk's two kinds of boxes, the missing arrival is made here,
  // so that the phase completes with the bytes); then q
  if (x.tid == 0 && x.n_chunks > 0) {
    const volatile int* issued = reinterpret_cast<const volatile int*>(smem + kOffIssued);
    for (int e = 0; e < kVChunks; ++e) {
      const int k = issued[e], v = issued[kVChunks + e], c = max(k, v);
      if (c < 0) continue;
      if (k != v) mbar_arrive(x.bar(kFull + e));
      drain_wait(x, x.bar(kFull + e), (c / kVChunks) & 1, 12);
    }
    drain_wait(x, x.bar(kQFull), 0, 13);
  }
}

template <Keys KEYS, bool UNI>
cudaError_t launch_variant(const VsMaps& maps, const DecodeParams& p, dim3 grid, int* status, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(decode_vs_kernel<KEYS, UNI>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  decode_vs_kernel<KEYS, UNI><<<grid, kThreads, kSmem, stream>>>(maps, p, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_vs(const DecodeParams& p, int64_t q_rows, int64_t kv_rows, dim3 grid, int* status,
                             cudaStream_t stream) {
  if (p.kv_scales == nullptr) return cudaErrorInvalidValue;
  const bool boxes = p.slots == nullptr && p.block_size % kHalf == 0;
  VsMaps maps{};
  cudaError_t e = make_row_map(&maps.q, p.q, static_cast<uint64_t>(q_rows), kRows, true);
  if (e == cudaSuccess) e = make_row_map(&maps.qr, p.q, static_cast<uint64_t>(q_rows), kRows, true, 64);
  if (e == cudaSuccess && boxes) e = make_row_map(&maps.kv, p.kv, static_cast<uint64_t>(kv_rows), kHalf, true);
  if (e == cudaSuccess && boxes) e = make_row_map(&maps.kvr, p.kv, static_cast<uint64_t>(kv_rows), kHalf, true, 64);
  if (e == cudaSuccess && p.out != nullptr)
    e = make_out_map(&maps.out, p.out, static_cast<uint64_t>(q_rows), 1, true, 64, 32, true);
  if (e == cudaSuccess && p.segm_out != nullptr)
    e = p.items != nullptr
            ? make_out_map(&maps.part, p.segm_out, static_cast<uint64_t>(p.segm_rows), 1, false, 32, 32, true)
            : make_out_map(&maps.part, p.segm_out, static_cast<uint64_t>(q_rows),
                           static_cast<uint64_t>(p.num_segments), false, 32, 32, true);
  if (e != cudaSuccess) return e;
  if (p.slots != nullptr) return launch_variant<Keys::kList, false>(maps, p, grid, status, stream);
  if (!boxes) return launch_variant<Keys::kBlocks, false>(maps, p, grid, status, stream);
  // groups of a multiple of 16 slots: 16 keys from a 16-aligned position (of one
  // block) share their scale, and a softmax thread reads two for its 32 keys
  // instead of 32 (32 requests of 1 to 3 tokens, groups of 16: 97 against 90 us)
  return p.scale_group % kUni == 0 ? launch_variant<Keys::kBoxes, true>(maps, p, grid, status, stream)
                                    : launch_variant<Keys::kBoxes, false>(maps, p, grid, status, stream);
}

}  // namespace mla

// Attention of blocks of rows over the paged cache, bf16: 5th-generation
// tensor cores (the operator is described in sf_cache_rows.cu).
//
// A tile is up to 256 query vectors, two halves of 128 (a half's vectors are
// the 128 TMEM lanes), over blocks of 128 keys.  Per half and block
//   S = Q K^T   tcgen05.mma, Q and K from shared memory, S in TMEM
//   P = 2^(x - m - kRowsRoom) by one thread per vector, written over S as bf16
//   O += P V    tcgen05.mma, P from TMEM, V MN-major from shared memory, O in
//               TMEM
// and the two halves take turns: one's softmax runs while the tensor core works
// for the other.  A tile of one half alone ("narrow") gives both softmax groups
// the same vectors and every other block each; their two results meet in
// registers at the end.  Its bound is the keys' bandwidth, not the tensor core,
// so P enters there as the sum of two bf16 numbers.
//
// Order on the tensor core.  One thread issues all of a half's MMAs, and they
// execute in that order; a commit covers all before it.  S of a half's next
// block follows its O += P V (whose P it overwrites), so when the softmax sees
// the new S, O is at rest: a row whose maximum grows by more than kSlack
// rescales it there (rarely: the maximum is kept only to within 2^kSlack).
// Each half has an issuing warp of its own: a wait costs 110 cycles even where
// there is nothing to wait for, and the tensor core's queue is short (one warp
// for both took 3,700 cycles for a block of two halves).  The two issue in turns:
// left alone they fall into step, both softmaxes and then both products at once
// (4,200 cycles).  So a block of two halves takes some 3,000 cycles, 2,048 of
// them the tensor core's (128 dimensions): what is left is a half's softmax
// (1,690, of which 512 are the exponentials at 32 a cycle) and its products' round
// trips, a chain that two halves cannot hide altogether.  16 ragged sequences of
// up to 1,021 rows over up to 8,191 keys, 32/8 heads: 518 to 540 us a call (61 %
// of the cuBLAS rate); 4 of 288 rows over 4,096, 40/8 heads: 97 (52 %).  Scores of
// both halves in one region of TMEM, so that a half's next scores come before its
// product, take 2,700 cycles a block where the keys are in L2, but large calls are
// no faster (1,280 TFLOP/s back to back either way), 4 of 288 rows took 97 instead
// of 102 then, and a batch with shared prefixes 99 instead of 98.
//
// P enters the second product of a wide tile rounded to bf16, half a step of 2^-8
// a weight, the output type's own, in calls that give a thread block more than
// two of its blocks (kTcExact): the product for the remainder costs 16 ragged
// sequences of up to 1,021 rows 535 -> 700 us, 4 of 288 rows 102 -> 124, a ragged
// batch with shared prefixes 98 -> 112, 288 rows over 1,024 to 4,096 keys 10 to
// 18 %.  Smaller calls wait for latency, not the tensor core: P is the sum of two
// bf16 numbers there too, for 2 to 7 % (32 rows over 512 keys, 12/2 heads 15.2 ->
// 15.6 us; over 4,096 keys, 40/8 heads 20.4 -> 21.7).
//
// Warps: 0-3 softmax and epilogue of half 0, 4-7 of half 1, 8 and 9 the MMAs of
// the halves (8 owns TMEM), 10 keys, 11 values.  Warp 10 also walks along the
// block's share of the batch and hands the parts to the others through a ring.
// Loads are TMA.  An instruction costs the unit some 46 cycles and 2.6 for each
// 128 bytes (4, 8, 16, 32, 64, 128 rows of 64 dimensions: 8.5, 14.5, 22.5, 31,
// 38, 43 bytes a cycle and SM), so rows that follow one another in a page come
// in as large boxes as its size allows, whole heads at a time; rows at the seams
// of odd pages and behind the end four at a time (gather4), with zeros for
// positions that are not there.
#include <cmath>
#include <type_traits>

#include "sf_cache_rows.cuh"
#include "sf_internal.h"
#include "sf_pairs.cuh"
#include "sf_tc.cuh"

namespace sf {
namespace {

using namespace rows;

constexpr int kTcThreads = 384;
constexpr int kTcHalf = 128;   // query vectors of a half
constexpr int kTcKeys = 128;   // keys of a block
// Units of a tile, and of a block of it with one half and with two.
constexpr int kTcFixed = 24, kTcNarrow = 5, kTcWide = 6, kTcLeast = 6;
constexpr int kTcExact = 2 * kTcWide;  // units a thread block up to which wide tiles keep P as two numbers
constexpr int kLiveRing = 8;   // blocks whose masks of live keys are kept
constexpr float kSlack = 8.f;
constexpr int kMmaWarp = 8, kKeyWarp = 10, kValueWarp = 11;
constexpr int kPartRing = 4;

template <int HD>
struct TcLayout {
  static constexpr int ST = HD == 128 ? 2 : 4;       // stages of the key ring, and of the value ring
  // a stage: 128 rows in groups of eight, each 64 dimensions (1,024 bytes) after 64 dimensions
  static constexpr int HALVES = HD / 64, GROUP = HALVES * 1024, STAGE = 16 * GROUP;
  static constexpr int Q = 0;                        // two halves
  static constexpr int K = Q + 2 * STAGE;
  static constexpr int V = K + ST * STAGE;
  // rows on their way out: 64 bytes of 32 rows a warp, padded so that both ways meet few banks twice
  static constexpr int OUT = V + ST * STAGE, OUT_LD = 80, OUT_WARP = 32 * OUT_LD;
  static constexpr int BYTES = OUT + 8 * OUT_WARP + 1024;  // + alignment of the dynamic window
  static constexpr int O_COL = 256;                  // TMEM: S of half w at 128 w, O at 256 + HD w
  static_assert(BYTES <= 224 * 1024, "shared memory");
};

struct Barriers {
  uint64_t qfull[2], sfull[2], pfull[2][2], odone[2];  // of each half; P's in two parts of 64 keys
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t part_full[kPartRing], part_empty[kPartRing];
  uint64_t meet;  // of both softmax groups
  uint64_t turn[2];  // whose MMAs come next
  uint64_t drain[2];  // after a stall: a half's MMAs so far are done
};

// What a thread block does next: blocks b0 .. b0 + nb - 1 of a tile.
struct TcPart {
  int nb;        // 0: nothing more
  int wide;      // two halves
  int split;     // P as the sum of two bf16 numbers
  int nv;        // query vectors
  int kvh;
  int t0, rem;   // row and head (within the KV head) of its first vector
  int slot;      // of the partial result; -1: the tile is whole
  int s, len, b0;
};

// Waits are bounded.  One that gives up (limit_ns without its phase, or another
// wait of the block has given up) returns false, and the call is reported as
// stalled.  Who gets false leaves its loops there and then: it issues, loads,
// stores and arrives nothing more, so that a wait that returns true has seen
// what it waited for, and everybody else's waits end as well.  What is in flight
// by then, copies and products, is waited for at the end of the kernel.
struct Waits {
  volatile int* dead;
  unsigned* err;
  uint32_t limit_ns;

  template <typename Ready>
  __device__ __forceinline__ bool until(Ready ready) const {
    if (ready()) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    while (!ready()) {
      if (*dead) return false;
      if (tc::globaltimer_ns() - t0 > limit_ns) {
        *dead = 1;
        cache_error(err, kCacheStall);
        return false;
      }
    }
    return true;
  }
  __device__ __forceinline__ bool phase(uint64_t* bar, uint32_t parity) const {
    return until([&]() { return tc::mbar_try_wait(bar, parity); });
  }
  // The loads of block `b` of a ring have been issued.  A reader that skips
  // blocks (the other half's, in narrow tiles) may come to a stage two phases
  // early, where the phase's parity alone would let it through.
  __device__ __forceinline__ bool load(volatile uint32_t* issued, uint32_t b) const {
    return until([&]() { return *issued > b; });
  }
  // By whole warps, for copies and products, which end by themselves.
  __device__ __forceinline__ void drained(uint64_t* bar, uint32_t parity) const {
    const uint64_t t0 = tc::globaltimer_ns();
    while (!tc::mbar_try_wait(bar, parity) && tc::globaltimer_ns() - t0 < limit_ns) {
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Which of a part's blocks softmax group w takes: `n` of them, the i-th being
// block first + step * i of the part.
struct Share {
  int n, first, step;
};
__device__ __forceinline__ Share share_of(int nb, int wide, int w) {
  return wide ? Share{nb, 0, 1} : Share{(nb + 1 - w) >> 1, w, 2};
}

// Keys and values as rows for gather4, and as boxes of `run` rows: the largest
// power of two up to 128 that divides the page size, or 8 where that is less
// than 16 (any eight rows that follow one another then).
struct PoolMaps {
  CUtensorMap gather[2], box[2];
};

template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1) cache_rows_tc_kernel(const __grid_constant__ CacheRowsArgs a,
                                                                      const __grid_constant__ PoolMaps maps,
                                                                      const int run, const int q_sign) {
  using Lay = TcLayout<HD>;
  constexpr int ST = Lay::ST, CH = HD / 8;  // 16-byte chunks of a row
  extern __shared__ unsigned char smem_raw[];
  __shared__ Barriers bar;
  __shared__ TcPart ring_of_parts[kPartRing];
  __shared__ __align__(32) uint32_t live[kLiveRing][8];  // byte x: keys 4 x .. 4 x + 3
  __shared__ float2 sml[2][kTcHalf];
  __shared__ uint32_t tmem_slot;
  __shared__ int dead_;
  __shared__ volatile uint32_t issued[2];  // blocks of keys, of values
  const Waits waits{&dead_, a.err, a.wait_ns};
  unsigned char* base = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const RowsShape sh{a.group, a.nkv, kTcHalf, 2, kTcKeys, kTcFixed, {kTcNarrow, kTcWide}};

  if (tid == 0) {
    // an injected stall: one arrival more than there are, which nothing makes
    auto init = [&](uint64_t* b, int arrivals, CacheStallAt of) { tc::mbar_init(b, arrivals + (a.stall == of ? 1 : 0)); };
    for (int i = 0; i < 2; ++i) {
      init(&bar.qfull[i], kTcHalf, kStallQueries);
      init(&bar.sfull[i], 1, kStallScores);
      init(&bar.pfull[i][0], kTcHalf, kStallWeights);
      init(&bar.pfull[i][1], kTcHalf, kStallLateWeights);
      init(&bar.odone[i], 1, kStallOutputs);
      init(&bar.turn[i], 1, kStallTurn);
      tc::mbar_init(&bar.drain[i], 1);
    }
    for (int i = 0; i < ST; ++i) {
      init(&bar.kfull[i], 1, kStallKeys);
      init(&bar.kempty[i], 2, kStallKeysRead);  // both halves, or one of them twice
      init(&bar.vfull[i], 1, kStallValues);
      init(&bar.vempty[i], 2, kStallValuesRead);
    }
    for (int i = 0; i < kPartRing; ++i) {
      init(&bar.part_full[i], 1, kStallPart);
      init(&bar.part_empty[i], 11, kStallPartRead);  // 8 softmax warps, 2 issuers, values
    }
    init(&bar.meet, 2 * kTcHalf, kStallMeet);
    dead_ = 0;
    issued[0] = issued[1] = 0;
    tc::fence_barrier_init();
  }
  // before the next kernel may start: it could take the TMEM that this one would wait for
  if (warp == kMmaWarp) tc::tmem_alloc(&tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  if (!a.tail_ml) pdl_wait();  // beside the tail's kernel, which has waited for everything before it
  pdl_trigger();
  RowsWalk walk;
  bool empties;
  const bool ok = rows_plan<kTcThreads>(a, sh, walk, &empties);
  if (!ok) rows_refused(a);

  if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // the whole warp walks along, one lane issues: descriptors stay in uniform registers
    const bool leader = tc::elect_one();
    const int w = __shfl_sync(kFull, warp, 0) - kMmaWarp;
    const uint32_t idesc_s = tc::idesc_bf16_f32(kTcHalf, kTcKeys);
    const uint32_t idesc_o = tc::idesc_bf16_f32(kTcHalf, HD) | (1u << 16);  // V is MN-major
    const uint32_t base_u = __shfl_sync(kFull, tc::smem_u32(base), 0), tmem_u = __shfl_sync(kFull, tmem, 0);
    const uint64_t dq = tc::sw128_kmajor_desc(base_u + Lay::Q + w * Lay::STAGE, Lay::GROUP);
    const uint64_t dk = tc::sw128_kmajor_desc(base_u + Lay::K, Lay::GROUP);
    const uint64_t dv = tc::sw128_mnmajor_desc(base_u + Lay::V, 1024, Lay::GROUP);
    const uint32_t o_at = tmem_u + Lay::O_COL + w * HD, s_at = tmem_u + w * kTcKeys;
    auto waits_for = [&](uint64_t* b, uint32_t parity) { return __all_sync(kFull, waits.phase(b, parity)); };
    auto loaded = [&](int ring, uint32_t b, uint64_t* full) {
      return waits.load(&issued[ring], b) && waits.phase(full, (b / ST) & 1);
    };
    uint32_t blocks = 0, parts = 0, steps = 0, turns = 0;  // so far: of the rings, of this half
    for (uint32_t x = 0;; ++x) {
      if (!waits_for(&bar.part_full[x % kPartRing], (x / kPartRing) & 1)) break;
      const TcPart& p = ring_of_parts[x % kPartRing];
      const int nb = __shfl_sync(kFull, p.nb, 0), wide = __shfl_sync(kFull, p.wide, 0);
      const int split = __shfl_sync(kFull, p.split, 0);
      if (lane == 0) tc::mbar_arrive(&bar.part_empty[x % kPartRing]);
      if (nb == 0) break;
      const Share share = share_of(nb, wide, w);
      auto scores = [&](int i) {
        const uint32_t b = blocks + share.first + share.step * i, st = b % ST;
        if (!__all_sync(kFull, loaded(0, b, &bar.kfull[st]))) return false;
        tc::fence_after_sync();
        const uint64_t ka = dk + (uint64_t)((st * Lay::STAGE) >> 4);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4);
          tc::mma_bf16_by(leader, s_at, dq + off, ka + off, idesc_s, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit_by(leader, &bar.sfull[w]);
        tc::mma_commit_by(leader, &bar.kempty[st]);
        if (!wide) tc::mma_commit_by(leader, &bar.kempty[st]);
        return true;
      };
      if (share.n > 0) {
        if (!waits_for(&bar.qfull[w], parts & 1) || !scores(0)) break;
        ++parts;
      }
      int i = 0;
      for (; i < share.n; ++i, ++steps) {
        const uint32_t b = blocks + share.first + share.step * i, st = b % ST;
        const uint64_t va = dv + (uint64_t)((st * Lay::STAGE) >> 4);
        bool alive = loaded(1, b, &bar.vfull[st]) && waits.phase(&bar.pfull[w][0], steps & 1) &&
                     (!wide || waits.phase(&bar.turn[w], (turns & 1) ^ (w == 0 ? 1 : 0)));
        if (!__all_sync(kFull, alive)) break;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half && !(alive = waits_for(&bar.pfull[w][1], steps & 1))) break;
          tc::fence_after_sync();
#pragma unroll
          for (int kk = 4 * half; kk < 4 * half + 4; ++kk)  // 16 keys: two groups of V, 8 columns of P
            tc::mma_bf16_ts_by(leader, o_at, s_at + kk * 8, va + (uint64_t)((kk * 2 * Lay::GROUP) >> 4), idesc_o,
                               i > 0 || kk > 0 ? 1u : 0u);
          if (split)
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)  // what rounding P left
              tc::mma_bf16_ts_by(leader, o_at, s_at + 64 + kk * 8, va + (uint64_t)((kk * 2 * Lay::GROUP) >> 4), idesc_o, 1u);
        }
        if (!alive) break;
        tc::mma_commit_by(leader, &bar.vempty[st]);
        if (!wide) tc::mma_commit_by(leader, &bar.vempty[st]);
        if (i + 1 == share.n)
          tc::mma_commit_by(leader, &bar.odone[w]);
        else if (!scores(i + 1))
          break;
        if (wide) {
          if (leader) tc::mbar_arrive(&bar.turn[w ^ 1]);
          ++turns;
        }
      }
      if (i < share.n) break;
      blocks += nb;
    }
  } else if (warp == kKeyWarp || warp == kValueWarp) {
    // lane x takes keys 4 x .. 4 x + 3 of a block, and the box that starts there
    const bool keys = warp == kKeyWarp;
    const uint32_t ring =
        tc::smem_u32(base + (keys ? Lay::K : Lay::V)) + (lane >> 1) * Lay::GROUP + (lane & 1) * 512;
    uint64_t* full = keys ? bar.kfull : bar.vfull;
    uint64_t* empty = keys ? bar.kempty : bar.vempty;
    const CUtensorMap *gather = &maps.gather[keys ? 0 : 1], *box = &maps.box[keys ? 0 : 1];
    const int none = (int)(a.table.n_pages * a.table.page_size);  // a row outside the pool
    const int of_run = run / 4;                                   // lanes
    const unsigned peers = of_run == 32 ? kFull : ((1u << of_run) - 1u) << (lane / of_run * of_run);
    const bool leads = lane % of_run == 0;
    uint32_t blocks = 0;
    if (keys) {
      if (lane == 0) a.joins[blockIdx.x].n = 0;
      walk.start(sh);
    }
    for (uint32_t x = 0;; ++x) {
      TcPart& slot_of = ring_of_parts[x % kPartRing];
      if (keys) {  // the walk
        RowsPart p;
        SeqRows q;
        const bool more = walk.next(a, sh, p, q);
        const bool free = x < kPartRing || waits.phase(&bar.part_empty[x % kPartRing], (x / kPartRing - 1) & 1);
        if (!__all_sync(kFull, free)) break;  // nothing goes over a part that is still read
        if (lane == 0) {
          TcPart n{};
          if (more) {
            const int r = (int)quick_quotient(p.v0, a.group);
            n = TcPart{p.b1 - p.b0, p.w == 2, p.w == 1 || walk.per <= kTcExact, p.nv, p.kvh, q.row0 + r, p.v0 - r * a.group,
                       is_cut(p) ? rows_slot(blockIdx.x, p.b0 == 0) : -1, q.s, q.len, p.b0};
          }
          slot_of = n;
          tc::mbar_arrive(&bar.part_full[x % kPartRing]);
          if (more && is_cut(p) && p.b0 == 0) rows_record(a, p, q, walk.per);
        }
        __syncwarp();
      } else if (!__all_sync(kFull, waits.phase(&bar.part_full[x % kPartRing], (x / kPartRing) & 1))) {
        break;
      }
      const int nb = slot_of.nb, s = slot_of.s, len = slot_of.len, kvh = slot_of.kvh, b0 = slot_of.b0;
      __syncwarp();
      if (!keys && lane == 0) tc::mbar_arrive(&bar.part_empty[x % kPartRing]);
      if (__any_sync(kFull, nb == 0)) break;
      int32_t page[4];
      auto look = [&](int b) {  // page entries of this lane's keys of block b
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int j = b * kTcKeys + 4 * lane + t;
          page[t] = j < len ? entry_of(a, s, j) : -1;
        }
      };
      look(b0);
      int b = b0;
      for (; b < b0 + nb; ++b, ++blocks) {
        int slot[4];
        uint32_t there = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int j = b * kTcKeys + 4 * lane + t;
          slot[t] = none;
          if (j < len) {
            const uint32_t y = entry_slot32(a.table, page[t], j);
            if (y == ~0u)
              cache_error(a.err, kCacheBadPage);
            else
              slot[t] = (int)y, there |= 1u << t;
          }
        }
        if (b + 1 < b0 + nb) look(b + 1);
        // the lane's run is there and in one piece (runs from 16 on lie within a page)
        const int after = __shfl_down_sync(kFull, slot[0], 1);
        const bool joined = there == 15u && slot[3] == slot[0] + 3 && (run > 8 || (lane & 1) || after == slot[0] + 4);
        const bool whole = (__ballot_sync(kFull, joined) & peers) == peers;
        const uint32_t st = blocks % ST;
        const bool free = blocks < ST || waits.phase(&empty[st], (blocks / ST - 1) & 1);
        if (!__all_sync(kFull, free)) break;
        if (keys) reinterpret_cast<unsigned char*>(live[blocks % kLiveRing])[lane] = (unsigned char)there;
        __syncwarp();
        if (lane == 0) {
          tc::mbar_expect_tx(&full[st], Lay::STAGE);
          issued[keys ? 0 : 1] = blocks + 1;
        }
        __syncwarp();
        if (!whole) {
#pragma unroll
          for (int y = 0; y < HD / 64; ++y)
            tc::tma_gather4(ring + st * Lay::STAGE + y * 1024, gather, kvh * HD + 64 * y, slot[0], slot[1], slot[2],
                            slot[3], &full[st]);
        } else if (leads) {
          if (run == 8)
            tc::tma_load_4d(ring + st * Lay::STAGE, box, 0, slot[0], 0, kvh, &full[st]);
          else
            tc::tma_load_5d(ring + st * Lay::STAGE, box, 0, 0, 0, slot[0] >> 3, kvh, &full[st]);
        }
        __syncwarp();
      }
      if (b < b0 + nb) break;
    }
  } else {
    const int w = warp >> 2, r = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_at = lanes + w * kTcKeys, o_at = lanes + Lay::O_COL + w * HD;
    const float scale = a.scale_log2;
    const unsigned inverse = 0xffffffffu / (unsigned)a.group + 1u;  // (x inverse) >> 32 = x / group for x < 2^16, group > 1
    auto rows_in = [&](unsigned x) { return a.group == 1 ? x : __umulhi(x, inverse); };
    // Queries of part x, rows of 16-byte chunks, towards shared memory: this group's half (the S products of the part
    // before have read theirs).  A thread's chunks: column r % CH of rows r / CH, r / CH + 128 / CH, ...
    const uint32_t sq = tc::smem_u32(base + Lay::Q + w * Lay::STAGE);
    const int qc = r % CH, qr = r / CH;
    auto q_place = [&](int row) {
      return (row >> 3) * Lay::GROUP + (qc >> 3) * 1024 + (row & 7) * 128 + (((qc ^ row) & 7) << 4);
    };
    auto waits_for = [&](uint64_t* b, uint32_t parity) { return __all_sync(kFull, waits.phase(b, parity)); };
    auto there = [&](uint32_t x) { return waits_for(&bar.part_full[x % kPartRing], (x / kPartRing) & 1); };
    auto fetch_queries = [&](uint32_t x) {  // false: this group takes nothing of the part
      const TcPart& p = ring_of_parts[x % kPartRing];
      const int wide = p.wide, nv = p.nv - (wide ? w * kTcHalf : 0), t0 = p.t0, rem = p.rem + (wide ? w * kTcHalf : 0);
      if (share_of(p.nb, wide, w).n == 0) return false;
      const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)p.kvh * a.group * HD + qc * 8;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int row = qr + k * (128 / CH), v = rem + (row < nv ? row : 0), t = rows_in(v);
        const uint32_t to = sq + q_place(row);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                     "l"(from + (int64_t)(t0 + t) * a.ld_q + (v - t * a.group) * HD),
                     "r"(row < nv ? 16 : 0)
                     : "memory");
      }
      return true;
    };
    auto queries_there = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (q_sign <= 0) {
        const __nv_bfloat162 sign = __float2bfloat162_rn((float)q_sign);
        auto times = [&](uint32_t x) {  // exact; 0 times NaN or infinity is NaN
          const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), sign);
          return *reinterpret_cast<const uint32_t*>(&y);
        };
#pragma unroll 1
        for (int k = 0; k < CH; ++k) {
          const int row = qr + k * (128 / CH);
          uint4* u = reinterpret_cast<uint4*>(base + Lay::Q + w * Lay::STAGE + q_place(row));
          *u = make_uint4(times(u->x), times(u->y), times(u->z), times(u->w));
        }
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(&bar.qfull[w]);
    };
    uint32_t blocks = 0, steps = 0, parts = 0, meetings = 0;
    auto groups_meet = [&]() {  // not a bar.sync: a wait that ends
      tc::fence_before_sync();
      tc::mbar_arrive(&bar.meet);
      const bool ok = waits_for(&bar.meet, meetings & 1);
      ++meetings;
      tc::fence_after_sync();
      return ok;
    };
    bool alive = there(0);
    if (alive && fetch_queries(0)) queries_there();
    for (uint32_t x = 0; alive; ++x) {
      const TcPart& p = ring_of_parts[x % kPartRing];
      const int nb = p.nb, wide = p.wide;
      if (__any_sync(kFull, nb == 0)) break;
      const Share share = share_of(nb, wide, w);
      float m = -INFINITY, l = 0.f;
      auto step = [&](int i, auto split) {
        constexpr bool SPLIT = decltype(split)::value;  // P as two bf16 numbers
        const bool ok = waits.phase(&bar.sfull[w], steps & 1);
        __syncwarp();  // tensor-memory accesses are the whole warp's
        tc::fence_after_sync();
        const uint32_t* on = live[(blocks + share.first + share.step * i) % kLiveRing];
        const bool holes = on[lane >> 2] != 0x0f0f0f0fu;
        float s[128];
        tc::tmem_ld128(s_at, s);
        if (__any_sync(kFull, holes || !ok)) {
          if (__any_sync(kFull, !ok)) return false;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const uint32_t word = on[x];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (!(word >> (8 * (k >> 2) + (k & 3)) & 1)) s[16 * x + k] = -INFINITY;
          }
        }
        float t[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = s[k];
#pragma unroll
        for (int k = 4; k < 124; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = fmaxf(fmaxf(t[e], s[k + e]), s[k + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = fmaxf(t[e], s[124 + e]);
        const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale;
        const bool grew = top > m + kSlack;
        if (__any_sync(kFull, grew)) {  // the whole warp: TMEM accesses are collective
          const float to = grew ? top : m;
          if (i > 0) {
            const float f = grew ? ex2(m - to) : 1.f;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              float o[32];
              tc::tmem_ld32(o_at + c, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= f;
              tc::tmem_st32(o_at + c, o);
            }
          }
          m = to;
        }
        const float bias = (m == -INFINITY ? 0.f : -m) - kRowsRoom;
        const Two scale2 = two(scale, scale), bias2 = two(bias, bias);
        Two sum[2] = {two(0.f, 0.f), two(0.f, 0.f)};
        uint32_t hi[2][16], lo[16];
        auto weights = [&](int c) {  // keys 32 c .. of the block
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x = both(fma2(two(s[32 * c + 2 * k], s[32 * c + 2 * k + 1]), scale2, bias2));
            const float p0 = ex2(x.x), p1 = ex2(x.y);
            sum[k & 1] = sum[k & 1] + two(p0, p1);
            hi[c & 1][k] = pack_bf16(p0, p1);
            if constexpr (SPLIT)
              lo[k] = pack_bf16(p0 - __uint_as_float(hi[c & 1][k] << 16), p1 - __uint_as_float(hi[c & 1][k] & 0xffff0000u));
          }
          if constexpr (SPLIT) tc::tmem_st_u32<16>(s_at + 64 + 16 * c, lo);
        };
        auto store = [&](int c) { tc::tmem_st_u32<16>(s_at + 16 * c, hi[c & 1]); };
        auto arrive = [&](int half) {  // 64 keys: their product may begin
          tc::tmem_wait_st();
          tc::fence_before_sync();
          tc::mbar_arrive(&bar.pfull[w][half]);
        };
        // stores complete behind the next keys' exponentials
        weights(0);
        store(0);
        weights(1);
        store(1);
        weights(2);
        arrive(0);
        store(2);
        weights(3);
        store(3);
        arrive(1);
        const float2 x = both(sum[0] + sum[1]);
        l += x.x + x.y;
        ++steps;
        return true;
      };
      if (!p.split) {
#pragma unroll 1
        for (int i = 0; alive && i < share.n; ++i) alive = step(i, std::false_type());
      } else {
#pragma unroll 1
        for (int i = 0; alive && i < share.n; ++i) alive = step(i, std::true_type());
      }
      if (!alive) break;
      blocks += nb;
      // the next part's queries on their way, then on the tensor core while this part's results go out
      if (!(alive = there(x + 1))) break;
      const bool next = fetch_queries(x + 1);
      if (share.n > 0) {
        if (!waits_for(&bar.odone[w], parts & 1)) break;
        ++parts;
        tc::fence_after_sync();
      }
      if (next) queries_there();
      if (share.n > 0) {
        // columns [c0, c1) of the rows are this group's to finish
        const bool meet = !wide && nb > 1;  // the two groups' results do
        int c0 = 0, c1 = HD;
        float f0 = 1.f, f1 = 0.f;
        if (meet) {
          sml[w][r] = make_float2(m, l);
          if (!groups_meet()) break;
          const float2 y = sml[0][r], z = sml[1][r];
          const float top = fmaxf(y.x, z.x), b = top == -INFINITY ? 0.f : top;
          f0 = ex2(y.x - b);
          f1 = ex2(z.x - b);
          m = top;
          l = y.y * f0 + z.y * f1;
          c0 = w * (HD / 2);
          c1 = c0 + HD / 2;
        }
        const int row0 = wide ? w * kTcHalf : 0, row = row0 + r, slot = p.slot, nv = p.nv;
        const bool cut = slot >= 0, mine = row < nv;
        auto vector_at = [&](int row, int64_t* tr, int64_t* h) {  // row and head of a vector of the tile
          const unsigned v = p.rem + row, t = rows_in(v);
          *tr = p.t0 + (int64_t)t;
          *h = p.kvh * a.group + (int)(v - t * a.group);
        };
        int64_t tr, h;
        vector_at(row, &tr, &h);
        const int64_t at = tr * a.nq + h;
        float inv = 1.f;
        if (mine && c0 == 0) {
          if (cut) *part_ml<kTcTileRows>(a, slot, row) = make_float2(m, l);
          if (a.tail_ml) {
            if (!cut || p.b0 == 0) a.whole_ml[at] = make_float2(m, cut ? kRowCut : l);
          } else if (!cut && a.lse) {
            a.lse[at] = l == 0.f ? -INFINITY : kLn2 * (m + kRowsRoom) + logf(l);
          }
        }
        if (!cut && !a.tail_ml) inv = l == 0.f ? 0.f : 1.f / l;  // no score above -infinity: zeros
        f0 *= inv;
        f1 *= inv;
        // 64 bytes of each row through shared memory, so that four lanes write one row (a lane a row met a line each
        // with every store: 5,700 cycles a part)
        unsigned char* mem = base + Lay::OUT + warp * Lay::OUT_WARP;
        auto rows_out = [&](const uint4 (&u)[4], char* to, int64_t ld_t, int64_t ld_h) {
#pragma unroll
          for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(mem + lane * Lay::OUT_LD + 16 * k) = u[k];
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int x = (lane >> 2) + 8 * k, rx = row0 + 32 * (warp & 3) + x;
            int64_t tx, hx;
            vector_at(rx, &tx, &hx);
            if (rx < nv)
              *reinterpret_cast<uint4*>(to + tx * ld_t + hx * ld_h + (lane & 3) * 16) =
                  *reinterpret_cast<const uint4*>(mem + x * Lay::OUT_LD + (lane & 3) * 16);
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          float o[32];
          if (meet) {
            float y[32];
            tc::tmem_ld32(lanes + Lay::O_COL + c, o);
            tc::tmem_ld32(lanes + Lay::O_COL + HD + c, y);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = o[k] * f0 + y[k] * f1;
          } else {
            tc::tmem_ld32(o_at + c, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= f0;
          }
          if (cut) {
            if (mine)
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                *part_at<HD, kTcTileRows>(a, slot, (c + k) / 4, row) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            __syncwarp();  // the next loads are the whole warp's
          } else if (a.tail_ml) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint4 u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                u[k] = make_uint4(__float_as_uint(o[e + 4 * k]), __float_as_uint(o[e + 4 * k + 1]),
                                  __float_as_uint(o[e + 4 * k + 2]), __float_as_uint(o[e + 4 * k + 3]));
              rows_out(u, reinterpret_cast<char*>(a.whole_o + c + e), (int64_t)a.nq * HD * 4, HD * 4);
            }
          } else {
            uint4 u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              u[k] = make_uint4(pack_bf16(o[8 * k], o[8 * k + 1]), pack_bf16(o[8 * k + 2], o[8 * k + 3]),
                                pack_bf16(o[8 * k + 4], o[8 * k + 5]), pack_bf16(o[8 * k + 6], o[8 * k + 7]));
            rows_out(u, static_cast<char*>(a.out) + c * 2, a.ld_out * 2, HD * 2);
          }
        }
        if (meet && !groups_meet()) break;  // both O are read before either group lets the next part begin
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.part_empty[x % kPartRing]);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ok && (empties || a.tail_ml)) rows_empties<__nv_bfloat16, HD, 2 * kTcHalf>(a, empties);
  }
  if (a.tail_ml) pdl_wait();  // the join waits for this kernel only
  tc::fence_before_sync();
  __syncthreads();
  if (dead_) {  // nobody waits any more, so this is the same for all
    if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      tc::mma_commit_by(tc::elect_one(), &bar.drain[warp - kMmaWarp]);  // the same lane as ever
      waits.drained(&bar.drain[warp - kMmaWarp], 0);
    } else if (warp == kKeyWarp || warp == kValueWarp) {
      const uint32_t n = issued[warp - kKeyWarp];
      for (uint32_t b = n > ST ? n - ST : 0; b < n; ++b)
        waits.drained(&(warp == kKeyWarp ? bar.kfull : bar.vfull)[b % ST], (b / ST) & 1);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int HD>
cudaError_t rows_tc(cudaStream_t st, CacheRowsArgs a) {
  PoolMaps maps;
  const uint64_t slots = (uint64_t)a.table.n_pages * a.table.page_size;
  int run = 8;
  if (a.table.page_size % 16 == 0)
    while (run < kTcKeys && a.table.page_size % (2 * run) == 0) run *= 2;
  for (int i = 0; i < 2; ++i) {
    const void* pool = i ? a.v : a.k;
    if (!make_tmap_pool_rows(&maps.gather[i], pool, HD, a.nkv, slots) ||
        !make_tmap_pool_run(&maps.box[i], pool, HD, a.nkv, slots, run))
      return cudaErrorInvalidValue;
  }
  // a negative scale turns the queries' signs, 0 makes them 0 (NaN and infinite
  // ones NaN): the maximum of the scaled scores is then that of the scores
  const int sign = a.scale_log2 > 0.f ? 1 : a.scale_log2 < 0.f ? -1 : 0;
  a.scale_log2 = sign == 0 ? 1.f : fabsf(a.scale_log2);
  a.least = kTcLeast;
  return launch_pdl(st, dim3(a.ctas), dim3(kTcThreads), TcLayout<HD>::BYTES, 1, cache_rows_tc_kernel<HD>, a, maps, run,
                    sign);
}

}  // namespace

cudaError_t prepare_cache_rows_tc() {
  cudaError_t e = cudaFuncSetAttribute(cache_rows_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       TcLayout<128>::BYTES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(cache_rows_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcLayout<64>::BYTES);
  return e;
}

cudaError_t launch_cache_rows_tc(cudaStream_t st, const CacheRowsArgs& a, int hd) {
  return hd == 128 ? rows_tc<128>(st, a) : rows_tc<64>(st, a);
}

}  // namespace sf

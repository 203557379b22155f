"""How a batch's attention is split over thread blocks: the rules that the
kernel uses (csrc/sf_cache_index.h, compiled here as plain C++), block by
block, checked for any batch (CPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WARPS, THREADS = 8, 256        # of an attention block


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    src = d / "split.cpp"
    src.write_text("""
#include <algorithm>
#include <vector>
#include "sf_cache_index.h"
using namespace sf;
struct Part { int block, segment, t0, end, n, b0, slot0, slot; };

extern "C" {
// The parts of segments that the blocks of a launch take, in block order; returns how many, or ~that for chunks.
int split(const int* tiles, int S, int H, int blocks, int warps, int threads, Part* out) {
  Part* p = out;
  std::vector<int> first(S + 1, 0);
  int filled = 0;
  for (int s = 0; s < S; ++s) {
    first[s + 1] = first[s] + tiles[s];
    filled += tiles[s] > 0;
  }
  const long long units = (long long)first[S] * H;
  if (units == 0) return 0;
  const long long share = units_per_block(units, blocks, kLeast);
  if ((long long)filled * H <= blocks && S <= threads) {
    int size = (int)share, chunks = 0, longest = 0;
    for (int i = 0; i < kPlanTries; ++i) {
      chunks = longest = 0;
      for (int s = 0; s < S; ++s) {
        const int n = chunks_of(tiles[s], size);
        chunks += n;
        if (n) longest = std::max(longest, chunk_tiles(tiles[s], n));
      }
      if (chunks * H <= blocks) break;
      size = wider_chunks(size, chunks * H, blocks);
    }
    if (plan_fits(chunks * H, longest, share, blocks)) {
      int blk = 0;
      for (int s = 0; s < S; ++s)
        for (int hs = 0; hs < H; ++hs) {
          const int n = chunks_of(tiles[s], size);
          for (int x = 0; x < n; ++x, ++blk) {
            const int each = chunk_tiles(tiles[s], n);
            *p++ = Part{blk, s * H + hs, std::min(tiles[s], x * each), std::min(tiles[s], (x + 1) * each), n, blk - x,
                        2 * (blk - x), 2 * blk};
          }
        }
      return ~(int)(p - out);
    }
  }
  for (int blk = 0; blk < blocks; ++blk) {
    long long u = blk * share;
    const long long u_end = std::min(u + share, units);
    if (u >= u_end) continue;
    int s = 0;
    while ((long long)first[s + 1] * H <= u) ++s;
    const int in_s = (int)(u - (long long)first[s] * H);
    int hs = in_s / tiles[s], t0 = in_s % tiles[s];
    auto advance = [&]() {
      if (++hs == H) {
        hs = 0;
        do ++s;
        while (s < S && tiles[s] == 0);
      }
    };
    if (const int skip = skipped(t0, tiles[s])) {
      u += skip;
      t0 = 0;
      advance();
    }
    while (u < u_end) {
      if (tiles[s] <= kShort) {  // a warp each, up to `warps` of those that start in this block's units
        const long long left = std::min(u_end - u, (long long)warps * kShort);
        int n = 0, taken = 0;
        while (n < warps && taken < left && s < S && tiles[s] <= kShort) {
          *p++ = Part{blk, s * H + hs, 0, tiles[s], 1, blk, part_slot(blk, u + taken, share),
                      part_slot(blk, u + taken, share)};
          ++n;
          taken += tiles[s];
          advance();
        }
        u += taken;
        continue;
      }
      const long long seg0 = u - t0;
      const LineTake x = take_of_line(blk, u, u_end, t0, tiles[s], share);
      *p++ = Part{blk, s * H + hs, t0, x.end, x.b1 - x.b0 + 1, x.b0, part_slot(x.b0, seg0, share),
                  part_slot(blk, seg0, share)};
      u += x.end - t0;
      t0 = 0;
      advance();
    }
  }
  return (int)(p - out);
}
int blocks_of(long long units, int most) { return attend_blocks(units, most); }
int join_of(int longest, int heads, int blocks) { return may_need_join(longest, heads, blocks); }
int constants(int i) { const int c[4] = {kShort, kLeast, kInlineParts, kWaste}; return c[i]; }
}
""")
    so = d / "split.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "sparse_reuse_gb300", "csrc"), str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def _split(lib, tiles, H, blocks):
    t = np.asarray(tiles, np.int32)
    out = np.zeros((blocks + H * len(t) + 2 * blocks, 8), np.int32)
    n = lib.split(t.ctypes.data_as(ctypes.c_void_p), len(t), H, blocks, WARPS, THREADS,
                  out.ctypes.data_as(ctypes.c_void_p))
    return out[:~n if n < 0 else n], n < 0


def _check(lib, parts, tiles, H, blocks, chunks):
    """Every tile once; a segment's blocks agree on how many they are and where the
    first one's partial result is; no two cut segments share a slot or a counter;
    what the join in place and the join kernel look for is there; on a line, short
    segments are whole."""
    short, _, inline, _ = (lib.constants(i) for i in range(4))
    by_segment = {}
    for p in parts.tolist():
        by_segment.setdefault(p[1], []).append(p)
    assert sorted(by_segment) == [s * H + h for s in range(len(tiles)) if tiles[s] for h in range(H)]
    slots, counters, joined = set(), set(), []
    for seg, ps in by_segment.items():
        want = tiles[seg // H]
        at = 0
        for x, (block, _, t0, end, n, b0, slot0, slot) in enumerate(ps):
            assert t0 == at and end >= t0 and n == len(ps) and b0 == ps[0][0] and block == b0 + x < blocks
            assert slot0 == ps[0][7] and slot == (slot0 if x == 0 else 2 * (b0 + x)) and 0 <= slot < 2 * blocks
            at = end
            if n > 1:
                assert slot not in slots
                slots.add(slot)
        assert at == want and (chunks or len(ps) == 1 or want > short)
        if len(ps) > 1:
            assert ps[0][5] not in counters
            counters.add(ps[0][5])
        if len(ps) > inline:
            joined.append(ps[0][5])
            assert lib.join_of(max(tiles), H, blocks)
    for window in range(0, blocks, inline):
        assert sum(window <= b < window + inline for b in joined) <= 1


KINDS = ["any", "even", "one long", "short", "mostly empty", "about short"]


@pytest.mark.parametrize("seed", range(120))
def test_every_tile_is_taken_once(lib, seed):
    rng = np.random.default_rng([seed, 31])
    kind = KINDS[seed % len(KINDS)]
    S = int(np.exp(rng.uniform(0, np.log(600))))
    H = int(rng.choice([1, 2, 4, 7, 8, 40]))
    top = int(np.exp(rng.uniform(0, np.log(16384))))
    if kind == "even":
        tiles = np.full(S, top)
    elif kind == "one long":
        tiles = rng.integers(0, 5, S)
        tiles[rng.integers(S)] = top
    elif kind == "short":
        tiles = rng.integers(0, 16, S)
    elif kind == "mostly empty":
        tiles = rng.integers(1, top + 1, S) * (rng.random(S) < 0.1)
    elif kind == "about short":
        tiles = rng.integers(14, 20, S)
    else:
        tiles = rng.integers(0, top + 1, S)
    tiles = tiles.tolist()
    for most in (152, 148, 1, 17):
        blocks = lib.blocks_of(ctypes.c_longlong(S * H * max(1, max(tiles))), most)
        assert 1 <= blocks <= most
        parts, chunks = _split(lib, tiles, H, blocks)
        _check(lib, parts, tiles, H, blocks, chunks)


@pytest.mark.parametrize("tiles,H,chunks", [
    ([256] * 4, 8, True), ([8192], 4, True), ([16384], 1, True), ([1], 1, True), ([0, 5, 0], 2, True),
    ([4000, 1, 1], 8, True), ([60] * 19, 8, True), ([60] * 20, 8, False), ([3] * 300, 4, False),
    ([16] * 152, 1, True), ([17, 16, 15, 400] * 100, 2, False), ([16384] * 256, 8, False)])
def test_both_ways_of_splitting(lib, tiles, H, chunks):
    """Batches that get a block for every chunk, and batches on a line: each way is
    met, and right."""
    blocks = lib.blocks_of(ctypes.c_longlong(len(tiles) * H * max(tiles)), 152)
    parts, got = _split(lib, tiles, H, blocks)
    assert got == chunks
    _check(lib, parts, tiles, H, blocks, got)


def test_the_check_sees_what_goes_wrong(lib):
    """A split with a tile left out, taken twice, with a wrong count, or with two
    segments in one slot does not pass."""
    tiles, H = [900, 3, 700, 16, 17], 3
    parts, chunks = _split(lib, tiles, H, 152)
    _check(lib, parts, tiles, H, 152, chunks)
    cut = [i for i in range(len(parts)) if parts[i][4] > 1]
    for row, col, by in ((cut[3], 2, 1), (cut[3], 3, 1), (cut[3], 4, 1), (cut[3], 5, 1), (cut[0], 6, 1),
                         (cut[-1], 7, -2)):
        wrong = parts.copy()
        wrong[row, col] += by
        with pytest.raises(AssertionError):
            _check(lib, wrong, tiles, H, 152, chunks)
    with pytest.raises(AssertionError):
        _check(lib, np.delete(parts, cut[2], 0), tiles, H, 152, chunks)

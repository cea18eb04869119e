// How the workgroups of an attention over a paged cache find their rows and keys (paged_chunk.hip, paged_step.hip and the
// join in paged.hip).
//
// A request's rows are taken R tokens at a time, each with Gt query heads of one cache head: a row tile of up to M rows.
// Its keys are tiles of KT, in the order first keys, window (one run without a window).  Where the row tiles are too few to
// fill the machine, the tiles of a row tile's keys are divided over several workgroups, whose results a second kernel
// joins.  Lengths are known on the device only, so every workgroup works the division out for itself, from all of them,
// and finds its own item by a prefix sum over the requests: the items come out equal whatever the lengths are, and a
// captured launch takes new ones.  64 requests cost a workgroup about 1 us, and more of them as much for each 64 and, in
// chunks, each number of parts that is tried (plan_paged has both sides).  Undivided launches find their request by a search
// in cu_q instead.
#pragma once
#include "common.h"
#include "paged.h"

namespace idx {

struct Request {
  int32_t from, n, len;   // rows [from, from + n), the last of len keys
};
__device__ __forceinline__ Request request(const PagedArgs &a, int b) {
  Request r;
  r.from = min(max(a.cu_q[b], 0), a.T);
  r.n = min(max(a.cu_q[b + 1], r.from), a.T) - r.from;
  r.len = min(max(a.len_k[b], 0), a.max_len);
  return r;
}

// Key tiles of the rows row0 .. row0 + R - 1 of a request.
struct KeyTiles {
  int32_t hi;      // one past the last key that a row sees
  int32_t firsts;  // tiles of first keys, from key 0
  int32_t base;    // key at which the tile after them starts
  int32_t count;
};
template <int KT>
__device__ __forceinline__ KeyTiles key_tiles(const PagedArgs &a, const Request &r, int32_t row0, int32_t R) {
  KeyTiles k{0, 0, 0, 0};
  const int32_t p0 = r.len - r.n + row0, p1 = r.len - r.n + min(row0 + R, r.n) - 1;
  if (p1 < 0) return k;
  k.hi = p1 + 1;
  const int64_t low = a.window ? (int64_t)p0 - a.window + 1 : 0;
  const int32_t lo = low > 0 ? (int32_t)(low / KT) : 0;   // tile of the first row's window
  k.firsts = (int32_t)(((int64_t)min((int64_t)a.first, (int64_t)lo * KT) + KT - 1) / KT);
  k.base = lo * KT;
  k.count = k.firsts + (k.hi - 1) / KT + 1 - lo;   // (hi may be up to 2^31 - 1)
  return k;
}

struct Item {
  Request r;
  int32_t b;
  int32_t row0;            // first row of the tile, within the request
  int32_t split, splits;
  int32_t first_item;      // of the tile's split 0
  int32_t next;            // items from one split of a tile to the next
};

// The same in scalar registers.
__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p) {
  const uint64_t x = (uint64_t)p;
  return (const uint8_t *)((uint64_t)(uint32_t)uniform((int32_t)(x >> 32)) << 32 | (uint32_t)uniform((int32_t)x));
}
__device__ __forceinline__ Item uniform(const Item &w) {
  return {{uniform(w.r.from), uniform(w.r.n), uniform(w.r.len)}, uniform(w.b),          uniform(w.row0), uniform(w.split),
          uniform(w.splits),                                     uniform(w.first_item), uniform(w.next)};
}

__device__ __forceinline__ int32_t wave_sum_i(int32_t x) { return (int32_t)wave_sum((uint32_t)x); }

enum Find { ITEM, TILE, ROW };

// The id-th item of the launch's list (or its id-th row tile, or the tile of row id); false: there is none.  Every lane of
// the wave calls it with the same id and gets the same answer.  TILE and ROW are for the join of divided launches, and take
// the division from the word that the launch's first items left.
template <int KT, bool CHUNK, Find BY>
__device__ __forceinline__ bool find_item(const PagedArgs &a, uint32_t id, Item &w) {
  const int lane = threadIdx.x & 63;
  const int32_t R = a.R;
  w.split = 0;
  w.splits = 1;
  w.first_item = (int32_t)id;
  w.next = 0;
  if (!a.divide) {
    // request b's tiles are numbered from cu_q[b] / R + b on: that is at least as many numbers as it has tiles
    int lo = 0, count = a.B;
    while (count > 1) {
      const int step = (count + 63) / 64, at = lane * step;
      const bool ok = at < count && (uint32_t)(min(max(a.cu_q[lo + at], 0), a.T) / R + lo + at) <= id;
      const uint64_t m = __ballot(ok);
      const int k = m ? 63 - __builtin_clzll(m) : 0;
      lo += k * step;
      count = min(step, count - k * step);
    }
    w.b = lo;
    w.r = request(a, lo);
    const int64_t t = (int64_t)id - (w.r.from / R + lo);
    if (t < 0 || t * R >= w.r.n) return false;
    // the last rows, which see the most keys, first
    const int32_t nt = (w.r.n + R - 1) / R;
    w.row0 = (nt - 1 - (int32_t)t) * R;
    return true;
  }
  // The lane's request of 64, its row tiles and their key tiles; the first 64 are loaded once
  struct Mine {
    Request r;
    int32_t nt, c;
  };
  auto load = [&](int b0) {
    Mine x{{0, 0, 0}, 0, 0};
    if (b0 + lane < a.B) {
      x.r = request(a, b0 + lane);
      x.nt = (x.r.n + R - 1) / R;
      if (x.nt) x.c = key_tiles<KT>(a, x.r, (x.nt - 1) * R, R).count;
    }
    return x;
  };
  uint32_t left = 1;       // the division that the launch's first items left, requested beside the lengths
  if constexpr (BY != ITEM) left = *a.chunk;
  const Mine mine0 = load(0);
  if (!left) return false; // nothing is divided
  auto at = [&](int b0) { return b0 ? load(b0) : mine0; };
  auto parts = [&](const Mine &x, int32_t size) { return max((x.c + size - 1) / size, 1); };
  int32_t chunk;           // key tiles of an item at most
  if constexpr (BY != ITEM) {
    chunk = (int32_t)left;
  } else {
    // what the launch has to do, in key tiles
    const int32_t mu = a.Hkv * a.blocks;
    float total = 0.f;   // as the division needs it: no more exact than it is
    int32_t most = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
      const Mine x = at(b0);
      total += wave_reduce_f32((float)x.nt * (float)x.c, [](float y, float z) { return y + z; });
      most = max(most, (int32_t)wave_max((uint32_t)x.c));
    }
    const float share = total * (float)mu / (float)a.slots;
    // Lists that are nearly equal, one to a slot: left whole.  Others in half a slot's share at most, so that the last ones to
    // start end soon after the others (64 requests x 8 cache heads, 4100 keys each: 192 us whole, 203 in halves; 32 of 1600 to
    // 16384 keys, E4M3: 161 us in halves, 187 in whole shares).
    chunk = max((int32_t)__builtin_fminf(0.5f * share, 0x1p30f) + 1, a.min_tiles);
    if (!CHUNK && (float)most <= 1.25f * share) chunk = most;
    chunk = max(chunk, 1);
    if constexpr (CHUNK) {
      // Few and long items: the longest list in as many parts, up to 16, as would be through first.  Equal items run in rounds of
      // `slots`; unequal ones end within one item of an even share.  An item takes about 5 tiles' time besides its tiles, and
      // a division 4 for the partial outputs and the join.
      int64_t best = (int64_t)1 << 62;
      chunk = max(most, 1);
      for (int s = 1; s <= 16; s += s < 4 ? 1 : 2) {
        const int32_t size = max((most + s - 1) / s, 1);
        if (s > 1 && size < a.min_tiles) break;
        int32_t items = 0;
        for (int b0 = 0; b0 < a.B; b0 += 64) {
          const Mine x = at(b0);
          items += wave_sum_i(x.nt * parts(x, size));
        }
        if (s > 1 && (int64_t)items * mu > a.max_items) break;
        const int64_t rounds = ((int64_t)items * mu + a.slots - 1) / a.slots;
        const int64_t even = rounds * (size + 5);
        const int64_t uneven = (int64_t)(share + 5.f * (float)items * (float)mu / (float)a.slots) + size;
        const int64_t t = min(even, uneven) + (s > 1 ? 4 * rounds : 0);
        if (t < best) {
          best = t;
          chunk = size;
        }
      }
    }
    // for the join; 0: it has nothing to do
    if (id == 0 && threadIdx.x == 0) *a.chunk = most > chunk ? (uint32_t)chunk : 0u;
  }
  int32_t items = 0, tiles = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const Mine x = at(b0);
    const int32_t ns = parts(x, chunk), its = x.nt * ns;
    const int32_t upto = (int32_t)wave_incl_scan((uint32_t)its);
    const int32_t tiles_upto = BY == TILE ? (int32_t)wave_incl_scan((uint32_t)x.nt) : 0;
    bool here;
    if constexpr (BY == ITEM) here = (int64_t)id < (int64_t)items + upto;
    if constexpr (BY == TILE) here = (int64_t)id < (int64_t)tiles + tiles_upto;
    if constexpr (BY == ROW) here = (int32_t)id >= x.r.from && (int32_t)id < x.r.from + x.r.n;
    const uint64_t m = __ballot(here);
    if (m) {
      const int k = __builtin_ctzll(m);
      const int32_t n = __builtin_amdgcn_readlane(x.nt, k);
      w.splits = __builtin_amdgcn_readlane(ns, k);
      w.r = {__builtin_amdgcn_readlane(x.r.from, k), __builtin_amdgcn_readlane(x.r.n, k), __builtin_amdgcn_readlane(x.r.len, k)};
      w.b = b0 + k;
      const int32_t before = items + __builtin_amdgcn_readlane(upto, k) - n * w.splits;
      int32_t tile = 0;      // counted from the request's end: the last rows, which see the most keys, first
      if constexpr (BY == ITEM) {
        w.split = n > 0 ? ((int32_t)id - before) / n : 0;
        tile = n > 0 ? ((int32_t)id - before) % n : 0;
      }
      if constexpr (BY == TILE) tile = (int32_t)id - (tiles + __builtin_amdgcn_readlane(tiles_upto, k) - n);
      if constexpr (BY == ROW) tile = n - 1 - ((int32_t)id - w.r.from) / R;
      // (bounds that are not ascending could count past 32 bits, or past the launch)
      if (n <= 0 || tile < 0 || tile >= n || w.split < 0 || w.split >= w.splits) return false;
      w.row0 = (n - 1 - tile) * R;
      w.first_item = before + tile;
      w.next = n;
      const int64_t last = BY == ITEM ? (int64_t)id : (int64_t)w.first_item + (int64_t)(w.splits - 1) * n;
      return w.first_item >= 0 && (last + 1) * a.Hkv * a.blocks <= a.max_items;
    }
    items += __builtin_amdgcn_readlane(upto, 63);
    if constexpr (BY == TILE) tiles += __builtin_amdgcn_readlane(tiles_upto, 63);
  }
  return false;
}

}  // namespace idx

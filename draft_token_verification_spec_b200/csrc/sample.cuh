// Drawing a token from a logit row (spec_sample) and a row's largest logits (spec_top_logits).
//
// Both need few of a row's entries: the kept set of a truncated distribution is a prefix of the
// entries in (value desc, id asc) order, and so are the top logits.
//   row_tile        one tile of a row per block (rowtile.cuh): each warp's maximum, the sum of its
//                   weights where the rule needs it, and a list of the tile's entries at or above
//                   a threshold that about j of them reach.
//   finish_row      one block per row (or, finish_short, a warp): the lists are complete above the
//                   largest of the thresholds; that pool, sorted, gives the kept set, and the draw
//                   or the output is taken from it.
//   *_deep_kernel   a cluster of eight larger blocks per row that the pool does not settle, from
//                   the whole row; it returns at once where there is none.
// While all blocks of a call fit on the GPU at once, one launch does it all, a cluster per row
// (row_kernel); beyond that a finishing block would hold the place of tiles (2,048 rows of 128,256
// took 1.4 times as long in one launch), and each step has its own.
// What bounds them: the tiles by instruction issue (top 64 of 2,048 x 128,256 bfloat16: 137 us, 3.8
// TB/s, 83% of the issue slots), the rest by latency (64 x 128,256, top-p 0.9: tiles 14, finishing 29,
// the deep kernel 3 us with no row left, 45 with one).
// Every choice is made on double weights exp((l - m) / T), as in the other sampling calls of the
// library, or on float32 sums whose error bound (sum_error) leaves no other outcome.
#pragma once

#include "rowtile.cuh"

namespace sv {

constexpr int kMaxJ = 256;      // largest j a tile aims at
constexpr int kPoolCap = 3136;  // entries a finishing block sorts: four blocks to an SM's shared memory
constexpr int kPoolAim = 960;   // entries aimed at when the kept set's size is unknown: pools of about
                                // 2,200, which hold most nuclei (a pool short of one costs 45 us)

// What one warp of a tile saw.
struct WarpPart {
  float m;      // largest entry (-inf: none; NaN: an entry is NaN or +inf)
  float s;      // sum of exp((x - m) / T) of float32 weights, where the row needs it
  float tau;    // entries >= tau are listed
  int32_t cnt;  // how many they are in the tile (more than the list holds: it is not complete);
                // greedy rows: the lowest id that holds m
};
static_assert(sizeof(WarpPart) == 16, "WarpPart is 16 bytes");

// What finishing leaves to the deep kernel: whether the row is its, the row's maximum, and for a
// nucleus that its pool holds but the float32 sum leaves open, the keys that the cut lies between
// (top logits: the two halves of the row's sum).
struct RowLeft {
  int32_t todo;
  float m;
  uint32_t lo, hi;  // (lo 0: nothing known)
};

struct TileJob {
  const void* logits;
  long long stride;  // entries from one row to the next
  int rows, V, n;    // n tiles to a row
  int blocks;        // and blocks, a cluster
  int cap;           // list entries to a tile
  int pool;          // pool entries to a row
  WarpPart* parts;             // [rows][n][kWarps]
  unsigned long long* lists;   // [rows][n][cap]: (key << 32) | ~id
  RowLeft* left;               // [rows]
};

struct SampleJob {
  TileJob t;
  const float* uniforms;
  float temp, top_p, min_p;    // for every row ...
  int top_k;
  const float* row_temp;       // ... or each row's own, where not NULL
  const int32_t* row_top_k;
  const float* row_top_p;
  const float* row_min_p;
  int32_t* tokens;
  float* probs;                // or NULL
};

struct TopJob {
  TileJob t;
  int k;
  float temp;
  Log2Scale c;
  int32_t* ids;     // [rows][k]
  float* values;    // [rows][k]
  float* lse;       // [rows] or NULL
};

// What a row's settings ask of its tiles.
struct RowAsk {
  float T;
  double iT;
  int K;          // entries top-k keeps; V where it keeps all
  double p, q;    // top-p (>= 1: off), min-p (0: off)
  bool bad;       // settings out of their ranges
  bool greedy;    // the argmax alone
  bool sum;       // the weights' sum over the whole row
  int j;          // entries each tile's list aims at; 0: no list; < 0: the exact kernel's row
  __device__ __forceinline__ bool interleaved() const { return j != 0; }
};

__host__ __device__ inline int list_aim(int want, int n) {
  // an even share of the row's `want` largest entries and 4 more, never more than all of them: two
  // to three times that many reach the tiles' largest threshold, which covers what interleaved tiles
  // differ by (of 200 rows each of eight kinds, none fell short)
  const int share = (want + n - 1) / n + 4;
  return want < share ? want : share;
}
// Entries a row's pool holds: six times what all its tiles aim at (twice that many reach the
// largest threshold where the tiles hold alike); `want` < 0 where it is not known beforehand.
inline int pool_cap(int want, int n) {
  if (want < 0) return kPoolCap;
  const int least = n == 1 ? 2048 : 1024, c = 6 * n * list_aim(want, n);
  return c < least ? least : (c > kPoolCap ? kPoolCap : c);
}
// Entries a tile's list holds: about four times what it aims at (1.1 j to 2 j entries reach the
// threshold where the warps hold alike, more where they do not), with room for equal values; the
// whole pool's for rows of one tile, whose warps hold adjacent ids.
__host__ __device__ inline int list_cap(int j, int n) {
  return n == 1 ? 2048 : (j <= 64 ? 256 : (j <= 128 ? 512 : 1024));
}

__device__ __forceinline__ RowAsk row_ask(const SampleJob& j, int row) {
  RowAsk a;
  a.T = j.row_temp ? j.row_temp[row] : j.temp;
  const int k = j.row_top_k ? j.row_top_k[row] : j.top_k;
  a.p = double(j.row_top_p ? j.row_top_p[row] : j.top_p);
  a.q = double(j.row_min_p ? j.row_min_p[row] : j.min_p);
  a.bad = !(a.T >= 0.0f && a.T < INFINITY) || !(a.p > 0.0) || !(a.q >= 0.0 && a.q <= 1.0);
  a.K = (k >= 1 && k < j.t.V) ? k : j.t.V;
  a.greedy = !a.bad && (a.T == 0.0f || a.K == 1);
  a.iT = 1.0 / double(a.T);
  const bool all = a.K == j.t.V;
  const bool plain = all && a.p >= 1.0 && a.q == 0.0;
  a.sum = !a.bad && !a.greedy && all && (a.p < 1.0 || a.q == 0.0);
  a.j = 0;
  if (!a.bad && !a.greedy && !plain) {
    a.j = list_aim(all ? kPoolAim : a.K, j.t.n);
    if (a.j > kMaxJ) a.j = all ? kMaxJ : -1;
  }
  return a;
}

__device__ __forceinline__ RowAsk row_ask(const TopJob& j, int) {
  RowAsk a;
  a.T = j.temp;
  a.iT = 1.0 / double(a.T);
  a.K = j.k;
  a.p = 1.0;
  a.q = 0.0;
  a.bad = a.greedy = false;
  a.sum = j.lse != nullptr;
  a.j = list_aim(j.k, j.t.n);
  return a;
}

// A value at or below every entry whose weight reaches min_p, in a row whose maximum is m.
__device__ __forceinline__ float min_p_floor(const RowAsk& a, float m) {
  const double t = double(m) + double(a.T) * log(a.q) * (1.0 + 1e-9) - fabs(double(m)) * 1e-14;
  return __double2float_rd(t);
}

__device__ __forceinline__ Log2Scale row_scale(const SampleJob&, const RowAsk& a) {
  return log2_scale_row(a.T);
}
__device__ __forceinline__ Log2Scale row_scale(const TopJob& j, const RowAsk&) { return j.c; }

// Relative error bound of a row's weight sum S (weights relative to the row's maximum) taken
// by the tiles, and of any part of it relative to S. A weight 2^-y is off by 2^-22 (ex2) and by
// 2^-23 y ln 2 (the roundings of x - m and of its scaling); the mean of y over the mass is the
// entropy in bits less log2 S, at most log2(V / S). A warp adds 2,048 weights in a tree of eleven
// levels, 2^-24 each, and the rest is summed in double.
constexpr double kErrEven = 2.4e-7 + 6.6e-7;  // relative to the part summed
constexpr double kErrDouble = 1e-8;
__device__ __forceinline__ double sum_error_spread(int V, double S) {  // of all parts together
  return 8.3e-8 * fmax(log2(double(V) / fmax(S, 1e-300)), 0.0);
}
__device__ __forceinline__ double sum_error(int V, double S) {
  return kErrEven + sum_error_spread(V, S) + kErrDouble;
}

// The smallest value of the type at or above x (entries compare with either alike).
template <typename T>
__device__ __forceinline__ float value_up(float x) {
  if constexpr (sizeof(T) == 4)
    return x;
  else
    return __bfloat162float(__float2bfloat16_ru(x));
}
// -inf in place of the vector's entries >= tau.
template <typename T>
__device__ __forceinline__ void drop_from(uint4& w, float tau) {
  uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (sizeof(T) == 4) {
      if (__uint_as_float(v[q]) >= tau) v[q] = 0xFF800000u;
    } else {
      const uint32_t on = __hge2_mask(Elem<__nv_bfloat16>::pair(v[q]), __float2bfloat162_rn(tau));
      v[q] = (v[q] & ~on) | (0xFF80FF80u & on);
    }
  }
  w = make_uint4(v[0], v[1], v[2], v[3]);
}

// Descending sort of one value per lane.
__device__ __forceinline__ float warp_sort_desc(float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int s = k >> 1; s > 0; s >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, s);
      const bool keep_max = ((lane & s) == 0) == ((lane & k) == 0);
      v = keep_max ? fmaxf(v, o) : fminf(v, o);
    }
  return v;
}

// The r-th largest (1 <= r <= 32) of two lists sorted over the lanes: the largest of
// min(x_i, y_{r-2-i}) over the splits of r into i + 1 of x and the rest of y, either alone too.
__device__ __forceinline__ float nth_of_two(float x, float y, int r) {
  const int lane = threadIdx.x & 31, o = r - 2 - lane;
  const float yo = __shfl_sync(0xffffffffu, y, o & 31);
  float c = -INFINITY;
  if (lane < r) c = o < 0 ? x : fminf(x, yo);
  if (lane == r - 1) c = fmaxf(c, y);
#pragma unroll
  for (int q = 16; q > 0; q >>= 1) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, q));
  return c;
}

struct TileSmem {
  uint4 tile[kTileVectors];  // this thread's vector u at u kThreads + threadIdx.x
  float max[kWarps], tau[kWarps];
  int cnt;
  uint16_t queue[kWarps][kTileVecs * 32];  // a warp's vectors that hold an entry to list
};

// The r-th largest (1 <= r <= 32) of the lanes' values: r rounds of taking the largest out, or for
// larger r a sort (a round takes 6 instructions, the sort 75).
__device__ __forceinline__ float nth_of_warp(float v, int r) {
  if (r > 8) return __shfl_sync(0xffffffffu, warp_sort_desc(v), r - 1);
  uint32_t key = f32_key(v), top = 0u;
#pragma unroll 1
  for (int i = 0; i < r; ++i) {
    top = __reduce_max_sync(0xffffffffu, key);
    const uint32_t who = __ballot_sync(0xffffffffu, key == top);
    if (int(threadIdx.x & 31) == __ffs(int(who)) - 1) key = 0u;
  }
  return f32_of_key(top);
}

// One tile, held in shared memory (five blocks an SM, against four with it in registers: 145
// against 162 us for top-64 of 2,048 rows of 128,256; six spill, 165 us): each warp's maximum,
// weight sum and list. The list's threshold is the j-th largest,
// or a little less, of the maxima of the tile's 256 threads (two maxima a thread when j > 128): at
// least j entries reach it, and of entries in random places about 1.1 j to 1.4 j. Each warp sorts
// its 32 (or 64) maxima by shuffles and gives its jw-th, jw = ceil(j / 8); the least of the eight is
// taken, behind the tile's only barrier. Warps with fewer than jw maxima above -inf (the tile ends,
// or a mask leaves few entries) stand aside where the others make up j; failing that, the warps'
// 4 jw-th count. No entry is compared twice but those of the few vectors that hold one to list.
// Top-p rows leave the listed entries out of the sum: the finishing block weighs them in double, so
// that the error of the float32 weights is that of the rest alone.
template <typename T, typename Job>
__device__ void row_tile(const Job& j, const RowAsk& a, const RowView<T>& rv, int row, int tile,
                         TileSmem& sm) {
  constexpr int P = Elem<T>::kPerVec;
  const int n = j.t.n, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool il = a.interleaved();
  fetch_tile(rv, il, tile, n, sm.tile);
  const TileRef w = {sm.tile + threadIdx.x};
  tile_arrived();
  VecMax<T> vm[kTileVecs], half[2];  // maxima of the vectors, and of the thread's two halves
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    vm[u].add(w[u], true);
    half[u / (kTileVecs / 2)].join(vm[u], u % (kTileVecs / 2) == 0);
  }
  const float h0 = half[0].value(), h1 = half[1].value();
  const float wm = warp_max_nan(fmax_nan(h0, h1));
  const bool bad = !(wm < INFINITY);  // NaN or +inf
  WarpPart part = {bad ? NAN : wm, 0.0f, -INFINITY, 0};
  const bool any = !bad && wm > -INFINITY;
  const bool later = a.sum && a.j > 0 && a.p < 1.0;  // the sum waits for the threshold
  auto weigh = [&]() {
    const Log2Scale c = row_scale(j, a);
    float f[kTileVecs];
#pragma unroll
    for (int u = 0; u < kTileVecs; ++u) f[u] = vec_exp_sum<T>(w[u], wm, c);
#pragma unroll
    for (int o = kTileVecs / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < o; ++u) f[u] += f[u + o];
    return warp_sum_f32(f[0]);
  };
  if (a.sum && !later && any) part.s = weigh();
  if (a.j > 0) {
    const int jw = (a.j + kWarps - 1) / kWarps;
    const float hm = fmaxf(h0, h1);
    const float t = a.j <= 128 ? nth_of_warp(hm, jw)
                               : nth_of_two(warp_sort_desc(h0), warp_sort_desc(h1), jw);
    if (lane == 0) {
      sm.max[warp] = any ? wm : -INFINITY;
      sm.tau[warp] = t;
      if (warp == 0) sm.cnt = 0;
    }
    __syncthreads();
    float tau = INFINITY, m = -INFINITY;
    int have = 0;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      m = fmaxf(m, sm.max[q]);
      if (sm.tau[q] > -INFINITY) {
        tau = fminf(tau, sm.tau[q]);
        ++have;
      }
    }
    if (have * jw < a.j) {  // (uniform)
      const int jw4 = min(4 * jw, 32);
      const float t4 = nth_of_warp(hm, jw4);
      __syncthreads();
      if (lane == 0) sm.tau[warp] = t4;
      __syncthreads();
      tau = INFINITY;
      have = 0;
#pragma unroll 1
      for (int q = 0; q < kWarps; ++q)
        if (sm.tau[q] > -INFINITY) {
          tau = fminf(tau, sm.tau[q]);
          ++have;
        }
      if (have * jw4 < a.j) tau = -INFINITY;
    }
    if (a.q > 0.0 && a.K == j.t.V)  // min-p drops what lies below, whatever top-p keeps
      tau = fmaxf(tau, __fadd_rd(m, a.T * (__logf(float(a.q)) - 1e-5f)));  // (below the floor)
    tau = value_up<T>(tau);
    part.tau = tau;
    if (any) {
      unsigned long long* list =
          j.t.lists + (size_t(row) * n + tile) * size_t(j.t.cap);
      uint32_t hit = 0u;
#pragma unroll
      for (int u = 0; u < kTileVecs; ++u)
        if (vm[u].reaches(tau)) hit |= 1u << u;
      // the warp's hit vectors in a queue, then an entry per lane, 32 / P vectors a round
      int at = __popc(hit);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += up;
      }
      const int hits = __shfl_sync(0xffffffffu, at, 31);
      at -= __popc(hit);
      for (; hit; hit &= hit - 1u)
        sm.queue[warp][at++] = uint16_t((__ffs(int(hit)) - 1) * 32 + lane);
      __syncwarp();
#pragma unroll 1
      for (int b = 0; b < hits; b += 32 / P) {
        const int i = b + lane / P;
        float x = -INFINITY;
        int id = 0;
        if (i < hits) {
          const int v = sm.queue[warp][i];
          id = rv.first(tile_vector_of(true, tile, n, v >> 5, warp, v & 31)) + lane % P;
          x = entry_of<T>(sm.tile[(v >> 5) * kThreads + warp * 32 + (v & 31)], lane % P);
        }
        const bool take = x >= tau && x > -INFINITY;
        const uint32_t mask = __ballot_sync(0xffffffffu, take);
        int base = 0;
        if (lane == 0) base = atomicAdd(&sm.cnt, __popc(mask));
        base = __shfl_sync(0xffffffffu, base, 0) + __popc(mask & ((1u << lane) - 1u));
        if (take && base < j.t.cap)
          list[base] = ((unsigned long long)f32_key(x) << 32) |
                       (unsigned long long)(0xFFFFFFFFu - uint32_t(id));
      }
      if (later) {
#pragma unroll
        for (int u = 0; u < kTileVecs; ++u) drop_from<T>(w[u], tau);
        part.s = weigh();
      }
    }
  } else if (a.greedy && any) {
    int id = INT_MAX;
#pragma unroll
    for (int u = 0; u < kTileVecs; ++u)
      if (vm[u].value() == wm) {
        float x[P];
        Elem<T>::unpack(w[u], x);
        const int e0 = rv.first(tile_vector(false, tile, n, u));
#pragma unroll
        for (int e = P - 1; e >= 0; --e)
          if (x[e] == wm) id = min(id, e0 + e);
      }
    part.cnt = __reduce_min_sync(0xffffffffu, id);
  }
  if (a.j > 0) {
    __syncthreads();
    part.cnt = sm.cnt;
  }
  if (lane == 0) j.t.parts[(size_t(row) * n + tile) * kWarps + warp] = part;
}

// ------------------------------------------------------------------------- finishing
constexpr int kSortBins = 1024;

// A finishing block's shared memory: this, then the pool and the sort's other buffer (later the
// weights), whose size the host chooses (pool_cap).
struct __align__(16) PoolSmem {
  __align__(16) uint32_t bins[kSortBins];
  int cap;  // entries of the pool
  __device__ __forceinline__ unsigned long long* e() {  // (key << 32) | ~id
    return reinterpret_cast<unsigned long long*>(this + 1);
  }
  __device__ __forceinline__ unsigned long long* tmp() { return e() + cap; }
  __device__ __forceinline__ double* w() { return reinterpret_cast<double*>(tmp()); }
  uint32_t lo, hi, crowd;
  double scr[kWarps];
  double tab[64];
  int cnt[kMaxTiles];
  float wm[kWarps], wtau[kWarps];
  float m;
  float tau;
  double s;
  int bad, over, n, best, cut;
};

inline size_t pool_bytes(int cap) {
  return sizeof(PoolSmem) + 2 * size_t(cap) * sizeof(unsigned long long);
}
static_assert(4 * (sizeof(PoolSmem) + 2 * kPoolCap * sizeof(unsigned long long) + 1024) <= 228 * 1024,
              "four finishing blocks to an SM");
__device__ __forceinline__ PoolSmem* pool_smem(int cap) {
  extern __shared__ __align__(16) unsigned char sv_pool[];
  PoolSmem* p = reinterpret_cast<PoolSmem*>(sv_pool);
  if (threadIdx.x == 0) p->cap = cap;  // (a barrier of finish_row stands before its first use)
  return p;
}

__device__ __forceinline__ int warp_of(int tid) { return tid >> 5; }

__device__ __forceinline__ float pool_value(unsigned long long e) {
  return f32_of_key(uint32_t(e >> 32));
}
__device__ __forceinline__ int pool_id(unsigned long long e) {
  return int(0xFFFFFFFFu - uint32_t(e & 0xFFFFFFFFull));
}

// Bitonic sort of the first N (a power of two) entries by the block.
template <bool kDesc, int kBlock>
__device__ __noinline__ void block_sort(unsigned long long* e, int N) {
#pragma unroll 1
  for (int k = 2; k <= N; k <<= 1)
#pragma unroll 1
    for (int s = k >> 1; s > 0; s >>= 1) {
#pragma unroll 1
      for (int i = threadIdx.x; i < N / 2; i += kBlock) {
        const int a = ((i & ~(s - 1)) << 1) | (i & (s - 1)), b = a | s;
        const unsigned long long x = e[a], y = e[b];
        const bool up = ((a & k) == 0) == kDesc;  // larger first
        if (up ? x < y : x > y) {
          e[a] = y;
          e[b] = x;
        }
      }
      __syncthreads();
    }
}
__device__ __forceinline__ int pow2_at_least(int n) {
  return n <= 1 ? 1 : 1 << (32 - __clz(n - 1));
}

// Sorts sm.e()[0..n) by the block: by value, larger first (kDesc, high words are keys), of which only
// the first `want` are wanted, or by id (high words are ids). The values (above -1e30: masks of the
// type's lowest value share the last range) or ids are cut into 1,024 equal ranges: counted, placed
// range by range, and ranked within their range by comparing with its other entries, which are
// few: seven barriers, against 78 of a bitonic network of 4,096. Where over 256 entries crowd into
// one range that is wanted (equal values), the network sorts instead. Ranges equal in the key would
// not do: from -5 to 8 they are 20 half-octaves (270 us instead of 20 for such a pool).
template <bool kDesc>
__device__ __noinline__ void pool_sort(PoolSmem& sm, int n, int want) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll 1
  for (int i = tid; i < n; i += kThreads) {
    const uint32_t h = uint32_t(sm.e()[i] >> 32);
    if (!kDesc || f32_of_key(h) > -1e30f) lo = min(lo, h);
    hi = max(hi, h);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (tid == 0) {
    sm.lo = 0xFFFFFFFFu;
    sm.hi = 0u;
    sm.crowd = 0u;
  }
  reinterpret_cast<uint4*>(sm.bins)[tid] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  if (lane == 0) {
    atomicMin(&sm.lo, lo);
    atomicMax(&sm.hi, hi);
  }
  __syncthreads();
  lo = sm.lo;
  hi = sm.hi;
  lo = min(lo, hi);
  const float base = kDesc ? f32_of_key(hi) : 0.0f;
  const float span = kDesc ? base - f32_of_key(lo) : float(hi - lo);
  const float scale = span > 0.0f ? float(kSortBins - 1) / span : 0.0f;
  // (each step rounds monotonously: ranges keep the order)
  auto bin = [&](unsigned long long x) {
    const uint32_t h = uint32_t(x >> 32);
    const float d = kDesc ? base - f32_of_key(h) : float(h - lo);
    return uint32_t(fminf(d * scale, float(kSortBins - 1)));
  };
#pragma unroll 1
  for (int i = tid; i < n; i += kThreads) atomicAdd(&sm.bins[bin(sm.e()[i])], 1u);
  __syncthreads();
  // each thread scans four bins; bins[] becomes where each starts
  const uint4 c = reinterpret_cast<uint4*>(sm.bins)[tid];
  const uint32_t own = c.x + c.y + c.z + c.w;
  uint32_t inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  uint32_t* wsum = reinterpret_cast<uint32_t*>(sm.scr);
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  uint32_t at = inc - own;
  for (int q = 0; q < warp; ++q) at += wsum[q];
  if (max(max(c.x, c.y), max(c.z, c.w)) > 256u && at < uint32_t(want)) sm.crowd = 1u;
  reinterpret_cast<uint4*>(sm.bins)[tid] = make_uint4(at, at + c.x, at + c.x + c.y, at + own - c.w);
  __syncthreads();
  if (sm.crowd) {
    const int N = pow2_at_least(n);  // (less than 2 n: it may reach into tmp())
    for (int i = n + tid; i < N; i += kThreads) sm.e()[i] = kDesc ? 0ull : ~0ull;
    __syncthreads();
    block_sort<kDesc, kThreads>(sm.e(), N);
    return;
  }
#pragma unroll 1
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long x = sm.e()[i];
    sm.tmp()[atomicAdd(&sm.bins[bin(x)], 1u)] = x;
  }
  __syncthreads();
  // now bins[b] is where range b ends, which is where range b + 1 starts
#pragma unroll 1
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long x = sm.tmp()[i];
    const uint32_t b = bin(x), b0 = b ? sm.bins[b - 1] : 0u, b1 = sm.bins[b];
    if (b0 >= uint32_t(want)) continue;
    uint32_t r = b0;
#pragma unroll 4
    for (uint32_t k = b0; k < b1; ++k) {
      const unsigned long long y = sm.tmp()[k];
      r += (kDesc ? y > x : y < x) ? 1u : 0u;
    }
    if (r < uint32_t(want)) sm.e()[r] = x;
  }
  __syncthreads();
}

// Row maximum, largest threshold, weight sum (of the float32 weights, when asked) and validity from
// the row's parts; every thread gets them through sm (barriers inside).
template <typename Job>
__device__ void merge_parts(const Job& j, const RowAsk& a, int row, PoolSmem& sm) {
  const int n = j.t.n * kWarps, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const WarpPart* parts = j.t.parts + size_t(row) * n;
  float m = -INFINITY, tau = -INFINITY;
  int bad = 0, over = 0;
#pragma unroll 1
  for (int i = tid; i < n; i += kThreads) {
    const WarpPart p = parts[i];
    bad |= !(p.m == p.m);
    m = fmaxf(m, p.m);
    if (a.j > 0) {
      if (p.m > -INFINITY) tau = fmaxf(tau, p.tau);
      if (p.cnt > j.t.cap) over = 1;
      if (i % kWarps == 0) sm.cnt[i / kWarps] = min(p.cnt, j.t.cap);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    tau = fmaxf(tau, __shfl_xor_sync(0xffffffffu, tau, o));
  }
  if (lane == 0) {
    sm.wm[warp] = m;
    sm.wtau[warp] = tau;
  }
  if (tid == 0) {
    sm.n = 0;
    sm.best = INT_MAX;
    sm.cut = INT_MAX;
  }
  bad = __syncthreads_or(bad);
  over = __syncthreads_or(over);
#pragma unroll
  for (int q = 0; q < kWarps; ++q) {
    m = fmaxf(m, sm.wm[q]);
    tau = fmaxf(tau, sm.wtau[q]);
  }
  if (tid == 0) {
    sm.m = m;
    sm.tau = tau;
    sm.bad = bad || !(m > -INFINITY);
    sm.over = over;
  }
  double s = 0.0;
  if (a.sum && !bad && m > -INFINITY) {
    const DoubleWeight f(m, a.iT, sm.tab);
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads) {
      const WarpPart p = parts[i];
      if (p.m > -INFINITY) s += double(p.s) * f(p.m);
    }
  }
  s = block_sum_f64(s, sm.scr);  // (barriers)
  if (tid == 0) sm.s = s;
  __syncthreads();
}

// Gathers the listed entries >= bound into sm.e; returns their number, or -1 when they do not fit.
// *mass, where given, gets this thread's share of the weights of the listed entries below bound.
__device__ __noinline__ int gather_pool(const TileJob& t, int row, float bound, PoolSmem& sm,
                                        double iT, double* mass) {
  const int n = t.n, tid = threadIdx.x, lane = tid & 31;
  const uint32_t key = f32_key(bound);
  const DoubleWeight f(sm.m, iT, sm.tab);
  double sum = 0.0;
  const unsigned long long* lists = t.lists + size_t(row) * n * size_t(t.cap);
  // eight tiles at a time, an entry of each per thread: their loads are under way together
  constexpr int kAt = 8;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kAt) {
    int most = 0;
#pragma unroll
    for (int q = 0; q < kAt; ++q) most = max(most, i0 + q < n ? sm.cnt[i0 + q] : 0);
#pragma unroll 1
    for (int b = 0; b < most; b += kThreads) {
      unsigned long long e[kAt];
#pragma unroll
      for (int q = 0; q < kAt; ++q)
        e[q] = i0 + q < n && b + tid < sm.cnt[i0 + q] ? lists[size_t(i0 + q) * t.cap + b + tid]
                                                      : 0ull;
      int own = 0;
#pragma unroll
      for (int q = 0; q < kAt; ++q) own += e[q] && uint32_t(e[q] >> 32) >= key ? 1 : 0;
      if (mass) {
#pragma unroll 1
        for (int q = 0; q < kAt; ++q) {
          if (i0 + q < n && b + tid < sm.cnt[i0 + q]) {
            const unsigned long long x = lists[size_t(i0 + q) * t.cap + b + tid];  // (in L1)
            if (uint32_t(x >> 32) < key) sum += f(pool_value(x));
          }
        }
      }
      int at = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += up;
      }
      int base = 0;
      if (lane == 31 && at) base = atomicAdd(&sm.n, at);
      at += __shfl_sync(0xffffffffu, base, 31) - own;
#pragma unroll
      for (int q = 0; q < kAt; ++q)
        if (e[q] && uint32_t(e[q] >> 32) >= key) {
          if (at < sm.cap) sm.e()[at] = e[q];
          ++at;
        }
    }
  }
  if (mass) *mass = sum;
  __syncthreads();
  const int c = sm.n;
  return c > sm.cap ? -1 : c;
}

// The lists are complete above the largest threshold, and the row needs entries below it: tiles that
// hold many of the largest entries have a high one. Adds the entries from `bound` up to their
// threshold from the tiles whose threshold lies above it (each read again by the whole block), so
// that sm.e, which holds the listed entries >= bound, is complete from bound on. Returns the number
// of entries, -1 when they do not fit.
template <typename T>
__device__ __noinline__ int complete_pool(const TileJob& t, const RowView<T>& rv, int row,
                                          float bound, PoolSmem& sm) {
  constexpr int P = Elem<T>::kPerVec;
  const int n = t.n;
  const WarpPart* parts = t.parts + size_t(row) * n * kWarps;
#pragma unroll 1
  for (int tile = 0; tile < n; ++tile) {
    // (a warp without an entry above -inf has no threshold; its fellows share one)
    float tau = -INFINITY;
    for (int q = 0; q < kWarps; ++q)
      if (parts[tile * kWarps + q].m > -INFINITY) tau = fmaxf(tau, parts[tile * kWarps + q].tau);
    if (!(tau > bound)) continue;
    uint4 w[kTileVecs];
    load_tile(rv, true, tile, n, w);
#pragma unroll 1
    for (int u = 0; u < kTileVecs; ++u) {
      float x[P];
      Elem<T>::unpack(w[u], x);
      const int e0 = rv.first(tile_vector(true, tile, n, u));
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (x[e] >= bound && x[e] < tau && x[e] > -INFINITY) {
          const int at = atomicAdd(&sm.n, 1);
          if (at < sm.cap)
            sm.e()[at] = ((unsigned long long)f32_key(x[e]) << 32) |
                       (unsigned long long)(0xFFFFFFFFu - uint32_t(e0 + e));
        }
    }
  }
  __syncthreads();
  const int c = sm.n;
  return c > sm.cap ? -1 : c;
}

// Leaves the row to the deep kernel (one thread calls).
__device__ __forceinline__ void leave_row(const TileJob& t, int row, float m, uint32_t lo = 0u,
                                          uint32_t hi = 0u) {
  t.left[row] = RowLeft{1, m, lo, hi};
}

__device__ __forceinline__ void write_draw(const SampleJob& j, int row, int tok, double w,
                                           double S) {
  j.tokens[row] = tok;
  if (j.probs) j.probs[row] = tok < 0 ? NAN : float(w / S);
}

// A plain draw (no truncation): the running sum of the parts' weights (a warp's 256 adjacent vectors
// each) finds the part, and its entries, read again by the block, the token.
template <typename T>
__device__ void plain_draw(const SampleJob& j, const RowAsk& a, const RowView<T>& rv, int row,
                           PoolSmem& sm) {
  constexpr int P = Elem<T>::kPerVec;
  const int n = j.t.n * kWarps, tid = threadIdx.x;
  const WarpPart* parts = j.t.parts + size_t(row) * n;
  const float m = sm.m;
  const double target = double(j.uniforms[row]) * sm.s;
  const DoubleWeight f(m, a.iT, sm.tab);
  constexpr int kMost = (kMaxTiles * kWarps + kThreads - 1) / kThreads;
  const int per = (n + kThreads - 1) / kThreads;
  double ps[kMost], own = 0.0, total;
#pragma unroll
  for (int q = 0; q < kMost; ++q) {
    const int i = tid * per + q;
    ps[q] = 0.0;
    if (q < per && i < n && parts[i].m > -INFINITY) ps[q] = double(parts[i].s) * f(parts[i].m);
    own += ps[q];
  }
  double cum = block_exclusive_scan(own, sm.scr, &total);
  // the first part whose running sum passes the target
  double c = cum;
#pragma unroll
  for (int q = 0; q < kMost; ++q) {
    c += ps[q];
    if (ps[q] > 0.0 && c > target) {
      atomicMin(&sm.cut, tid * per + q);
      break;
    }
  }
  __syncthreads();
  const int sel = sm.cut;
  if (sel == INT_MAX) {  // rounding or u >= 1
    if (tid == 0) leave_row(j.t, row, m);
    return;
  }
  if (sel / per == tid) {
    for (int q = 0; q < kMost; ++q)
      if (tid * per + q < sel) cum += ps[q];
    sm.w()[0] = cum;
  }
  __syncthreads();
  const double base = sm.w()[0];
  const int g = sel * (kTileVectors / kWarps) + tid;
  static_assert(kTileVectors / kWarps == kThreads, "one vector a thread");
  float x[P];
  Elem<T>::unpack(g < rv.G ? rv.load(g) : neg_inf_vec(int(sizeof(T))), x);
  double w[P];
  own = 0.0;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    w[e] = f(x[e]);
    own += w[e];
  }
  cum = base + block_exclusive_scan(own, sm.scr, &total);
  // An edge within `off` of the target leaves the row to the deep kernel. Where an edge has the mass B
  // before it and A after it, target less B is u A - (1 - u) B, off by at most kErrEven of
  // u A + (1 - u) B and max(u, 1 - u) of what the spread adds to all parts; u A + (1 - u) B is
  // linear in B and largest at one of this part's two ends. (Against 2 sum_error S: a quarter of
  // the rows.)
  const double S = sm.s, u = fmin(fmax(double(j.uniforms[row]), 0.0), 1.0);
  const double end = base + double(parts[sel].s) * f(parts[sel].m);
  const double mix = fmax(u * (S - base) + (1.0 - u) * base, u * (S - end) + (1.0 - u) * end);
  const double off =
      kErrEven * mix + (fmax(u, 1.0 - u) * sum_error_spread(j.t.V, S) + 2.0 * kErrDouble) * S;
  bool near = false;
  if (tid == 0) near = sel > 0 && !(target >= base + off);
  if (tid == kThreads - 1) near |= sel + 1 < n && !(target < cum + own - off);
  if (cum + own > target - off && cum <= target + off) {
    int best = INT_MAX;
    double e_cum = cum;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      e_cum += w[e];
      if (w[e] > 0.0) {  // (an entry without mass has no edge of its own)
        near |= fabs(e_cum - target) <= off;
        if (best == INT_MAX && e_cum > target) best = rv.first(g) + e;
      }
    }
    if (best != INT_MAX) atomicMin(&sm.best, best);
  }
  near = __syncthreads_or(near);
  if (tid == 0) {
    const int tok = sm.best;
    if (near || tok == INT_MAX)
      leave_row(j.t, row, m);
    else
      write_draw(j, row, tok, f(rv.entry(tok)), sm.s);
  }
}

// The kept prefix of the sorted pool sm.e()[0..c), complete down to `bound`: its length, or 0 when the
// row needs entries below the bound, or -1 when a decision lies within the sum's error. Z is the
// weights' total less the pool's for top-p (K == V) and off its error; every entry that min-p keeps
// is >= floor.
// sm.w gets the weights; sm.lo and sm.hi, with -1, where in the pool the cut lies between.
__device__ __noinline__ int kept_prefix(const RowAsk& a, int V, int c, float bound, float floor, double Z,
                           double off, PoolSmem& sm) {
  const int tid = threadIdx.x;
  const bool all = a.K == V;
  const int upto = min(c, a.K);
  const DoubleWeight f(sm.m, a.iT, sm.tab);
  const int per = (upto + kThreads - 1) / kThreads;
  const int i0 = tid * per, i1 = min(upto, i0 + per);
  double own = 0.0, total = 0.0;
  if (tid == 0) sm.cut = INT_MAX;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    const double w = f(pool_value(sm.e()[i]));
    sm.w()[i] = w;
    own += w;
  }
  const double before = block_exclusive_scan(own, sm.scr, &total);
  double cum = before;
  // (a bound of -inf: the pool is the row)
  const bool whole = bound == -INFINITY;
  if (!all && c < a.K && !whole) return 0;
  // top-k's first `upto`; of those, up to the entry whose running mass reaches top_p of the
  // total; of those, the ones whose weight reaches min_p
  const double reach = a.p * (all ? Z + total : total);
  bool near = false;
  int cut = INT_MAX;
#pragma unroll 1
  for (int i = i0; i < i1 && cut == INT_MAX; ++i) {
    const double w = sm.w()[i];
    cum += w;
    // (entry 0 is always kept: its weight is 1)
    if ((a.p < 1.0 && cum >= reach) || !(w > 0.0) || w < a.q)
      cut = (w > 0.0 && w >= a.q) ? i + 1 : i;
    // a running mass within the error of the total's: another entry may be the crossing one
    if (a.p < 1.0 && all && fabs(cum - reach) <= off + 1e-11 * cum && w > 0.0 && w >= a.q)
      near = true;
  }
  if (cut != INT_MAX) atomicMin(&sm.cut, cut);
  if (__syncthreads_or(near)) {
    // the first entries whose running mass may, and must, reach it: sm.lo and sm.hi
    if (tid == 0) sm.lo = sm.hi = 0xFFFFFFFFu;
    __syncthreads();
    cum = before;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      cum += sm.w()[i];
      if (cum >= reach - off - 1e-11 * cum) atomicMin(&sm.lo, uint32_t(i));
      if (cum >= reach + off + 1e-11 * cum) atomicMin(&sm.hi, uint32_t(i));
    }
    __syncthreads();
    return -1;
  }
  if (sm.cut != INT_MAX) return max(sm.cut, 1);
  // every pool entry is kept: the row's other entries have to be looked at, unless top-k ends
  // the kept set here, the pool is the whole row, or it holds all that min-p keeps
  if (all && !whole && !(a.q > 0.0 && bound <= floor)) return 0;
  return upto;
}

__device__ __forceinline__ void write_top(const TopJob& j, int row, int i, bool on,
                                          unsigned long long e) {
  j.ids[size_t(row) * j.k + i] = on ? pool_id(e) : -1;
  j.values[size_t(row) * j.k + i] = on ? pool_value(e) : -INFINITY;
}

// ------------------------------------------------------- the log-sum-exp of the top logits
// A list that holds all of a row's mass must not leave any over when its masses are taken with the
// row's log-sum-exp (the distillation loss would set it against a student that has none there). The
// float32 sum of the tiles is off by up to e = sum_error of itself. Where it exceeds the k largest,
// weighed in double, by more than 2 e there is mass outside them, and it stands. Else the sum is taken
// again, part by part (a warp's 256 vectors of a tile): the parts that hold more than 1 / (128
// parts) of it are read again, their entries among the k largest weigh in double, and only the rest
// of them in float32. The other parts are 1/128 of the sum together: it is off by e / 128 < 2.1e-8.
// Whether the sum stands, by the calling warp alone (all its lanes get the answer, every warp the
// same): float32 weights, off by less than 3e-6, tell most rows; e is under 2.6e-6. top: the `have`
// largest entries.
__device__ __forceinline__ bool sum_stands(const TopJob& j, double S, float m, double iT,
                                           const double* tab, const unsigned long long* top,
                                           int have) {
  const int lane = threadIdx.x & 31;
  float q = 0.0f;
#pragma unroll 1
  for (int i = lane; i < have; i += 32) q += weight_f(pool_value(top[i]), m, j.c);
  if (S - double(warp_sum_f32(q)) > 1e-5 * S) return true;
  const DoubleWeight f(m, iT, tab);
  double d = 0.0;
#pragma unroll 1
  for (int i = lane; i < have; i += 32) d += f(pool_value(top[i]));
  return S - warp_sum_f64(d) > 2.0 * sum_error(j.t.V, S) * S;
}

// The calling warp's share of that sum (each lane's is to be added): the parts and the k largest are
// dealt out to `warps` warps. top: the row's largest entries in order, `have` of them, fewer than k
// where no other is above -inf.
template <typename T>
__device__ __noinline__ double exact_share(const TileJob& t, const RowView<T>& rv, int row, float m,
                                           double iT, const double* tab, const Log2Scale& sc,
                                           const unsigned long long* top, int have, int k, double S,
                                           int warp, int warps) {
  constexpr int P = Elem<T>::kPerVec;
  const int n = t.n, parts_n = n * kWarps, lane = threadIdx.x & 31;
  const WarpPart* parts = t.parts + size_t(row) * parts_n;
  const DoubleWeight f(m, iT, tab);
  const double least = S / (128.0 * double(parts_n));
  auto mass = [&](int i) {
    const WarpPart p = parts[i];
    return p.m > -INFINITY ? double(p.s) * f(p.m) : 0.0;
  };
  double share = 0.0;
  const unsigned long long last = have >= k ? top[k - 1] : 0ull;
  const float b = pool_value(last);
#pragma unroll 1
  for (int i0 = warp * 32; i0 < parts_n; i0 += warps * 32) {
    const double w = i0 + lane < parts_n ? mass(i0 + lane) : 0.0;
    uint32_t again = __ballot_sync(0xffffffffu, w > least);
    if (!(w > least)) share += w;
    if (last == 0ull) continue;  // (the others' rests hold nothing)
#pragma unroll 1
    for (; again; again &= again - 1u) {
      const int i = i0 + __ffs(int(again)) - 1;
      uint4 v[kTileVecs];
#pragma unroll
      for (int u = 0; u < kTileVecs; ++u) {
        const int g = tile_vector_of(true, i / kWarps, n, u, i % kWarps, lane);
        v[u] = g < rv.G ? rv.load(g) : neg_inf_vec(int(sizeof(T)));
      }
      float s = 0.0f;
#pragma unroll
      for (int u = 0; u < kTileVecs; ++u) {
        float x[P], su = 0.0f;
        Elem<T>::unpack(v[u], x);
        const int e0 = rv.first(tile_vector_of(true, i / kWarps, n, u, i % kWarps, lane));
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const unsigned long long at = ((unsigned long long)f32_key(x[e]) << 32) |
                                        (unsigned long long)(0xFFFFFFFFu - uint32_t(e0 + e));
          if (x[e] > -INFINITY && at < last) su += weight_f(x[e], b, sc);
        }
        s += su;
      }
      s = warp_sum_f32(s);
      if (lane == 0) share += double(s) * f(b);
    }
  }
#pragma unroll 1
  for (int i = warp * 32 + lane; i < min(have, k); i += warps * 32) {
    const int piece = (pool_id(top[i]) + rv.mis) / P / 32;  // dealt out to the tiles in turn
    if (mass(piece % n * kWarps + piece / n % kWarps) > least) share += f(pool_value(top[i]));
  }
  return share;
}

__device__ __forceinline__ void write_lse(const TopJob& j, int row, float m, double iT, double S) {
  j.lse[row] = float(double(m) * iT + log(S));
}

// ------------------------------------------------------- finishing by one warp
// Rows that keep up to kShortK entries whatever the others weigh (spec_top_logits, one top-k for
// all rows): their pools are mostly under 256 entries, and a warp sorts those in its registers with
// no barrier, eight rows to a block. 2,048 rows of 128,256, top 64: 14.5 us, against 39 by a block
// each; the network's latency is longer than a block's (100 rows 12.4 against 9.2 us, 300 rows of
// top 128 14.1 against 10.1), so that it is taken for kShortRows rows and more, where not all
// blocks are on the GPU at once (512 rows 10.9 against 11.5, 600 rows 12.1 against 13.3). What does
// not fit (equal values, most of the largest in few warps' pieces) the block takes as above, row by
// row.
constexpr int kShortRows = 148 * 3;
constexpr int kShortK = 128;
constexpr int kShortPool = 256;
constexpr int kShortPer = kShortPool / 32;
constexpr int kShortRoom = 640;  // entries gathered; beyond kShortPool a higher bound is looked for

// Sorts e[0..256) by the calling warp, larger first: a bitonic network, eight adjacent entries a
// lane.
__device__ __noinline__ void warp_sort_pool(unsigned long long* e) {
  const int lane = threadIdx.x & 31;
  unsigned long long v[kShortPer];
#pragma unroll
  for (int r = 0; r < kShortPer; ++r) v[r] = e[lane * kShortPer + r];
  auto exchange = [](unsigned long long& x, unsigned long long& y, bool down) {
    const bool swap = (x < y) == down;
    const unsigned long long a = swap ? y : x, b = swap ? x : y;
    x = a;
    y = b;
  };
#pragma unroll
  for (int k = 2; k <= kShortPer; k <<= 1)
#pragma unroll
    for (int s = k >> 1; s > 0; s >>= 1)
#pragma unroll
      for (int r = 0; r < kShortPer; ++r)
        if (!(r & s))
          exchange(v[r], v[r | s], k == kShortPer ? (lane & 1) == 0 : (r & k) == 0);
#pragma unroll 1
  for (int k = 2; k <= 32; k <<= 1) {  // in lanes
    const bool down = (lane & k) == 0;
#pragma unroll 1
    for (int s = k >> 1; s > 0; s >>= 1) {
      const bool keep_max = ((lane & s) == 0) == down;
#pragma unroll
      for (int r = 0; r < kShortPer; ++r) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, v[r], s);
        v[r] = (v[r] < o) == keep_max ? o : v[r];
      }
    }
#pragma unroll
    for (int s = kShortPer / 2; s > 0; s >>= 1)
#pragma unroll
      for (int r = 0; r < kShortPer; ++r)
        if (!(r & s)) exchange(v[r], v[r | s], down);
  }
#pragma unroll
  for (int r = 0; r < kShortPer; ++r) e[lane * kShortPer + r] = v[r];
  __syncwarp();
}

__device__ __forceinline__ double warp_exclusive_scan(double own, double* total) {
  const int lane = threadIdx.x & 31;
  double inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  *total = __shfl_sync(0xffffffffu, inc, 31);
  return inc - own;
}

// The calling warp's row, its pool sorted in pool[0..256): true, with the row's maximum and (when asked)
// weight sum, where the pool holds the K largest.
template <typename Job>
__device__ __forceinline__ bool short_pool(const Job& j, const RowAsk& a, int row,
                                           unsigned long long* pool, const double* tab,
                                           float* max_, double* sum) {
  const int n = j.t.n, lane = threadIdx.x & 31;
  const WarpPart* parts = j.t.parts + size_t(row) * n * kWarps;
  float m = -INFINITY, tau = -INFINITY;
  bool stop = false;
#pragma unroll 1
  for (int i = lane; i < n * kWarps; i += 32) {
    const WarpPart p = parts[i];
    stop |= !(p.m == p.m) || p.cnt > j.t.cap;
    m = fmaxf(m, p.m);
    if (p.m > -INFINITY) tau = fmaxf(tau, p.tau);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    tau = fmaxf(tau, __shfl_xor_sync(0xffffffffu, tau, o));
  }
  if (__any_sync(0xffffffffu, stop) || !(m > -INFINITY)) return false;
  *max_ = m;
  // as gather_pool does
  const uint32_t key = f32_key(tau);
  const unsigned long long* lists = j.t.lists + size_t(row) * n * size_t(j.t.cap);
  constexpr int kAt = 8;
  int c = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kAt) {
    const int have = lane < kAt && i0 + lane < n ? parts[(i0 + lane) * kWarps].cnt : 0;
    const int most = __reduce_max_sync(0xffffffffu, have);
#pragma unroll 1
    for (int b = 0; b < most; b += 32) {
      unsigned long long e[kAt];
#pragma unroll
      for (int q = 0; q < kAt; ++q)
        e[q] = b + lane < __shfl_sync(0xffffffffu, have, q)
                   ? lists[size_t(i0 + q) * j.t.cap + b + lane] : 0ull;
#pragma unroll
      for (int q = 0; q < kAt; ++q) {
        const bool on = e[q] && uint32_t(e[q] >> 32) >= key;
        const uint32_t mask = __ballot_sync(0xffffffffu, on);
        const int at = c + __popc(mask & ((1u << lane) - 1u));
        if (on && at < kShortRoom) pool[at] = e[q];
        c += __popc(mask);
      }
    }
  }
  if (c > kShortRoom || c < a.K) return false;
  __syncwarp();
  if (c > kShortPool) {
    // a key that K to kShortPool entries reach, by halving the range of the keys
    uint32_t h[kShortRoom / 32];
#pragma unroll
    for (int q = 0; q < kShortRoom / 32; ++q)
      h[q] = q * 32 + lane < c ? uint32_t(pool[q * 32 + lane] >> 32) : 0u;
    uint32_t lo = key, hi = f32_key(m);  // lo: more than kShortPool; above hi: fewer than K
    int at = c;
    while (at > kShortPool && lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1u) / 2u;
      int own = 0;
#pragma unroll
      for (int q = 0; q < kShortRoom / 32; ++q) own += h[q] >= mid ? 1 : 0;
      const int reach = __reduce_add_sync(0xffffffffu, own);
      if (reach < a.K) {
        hi = mid - 1u;
      } else {
        lo = mid;
        at = reach;
      }
    }
    if (at > kShortPool) return false;  // (equal values)
    c = 0;
#pragma unroll
    for (int q = 0; q < kShortRoom / 32; ++q) {
      const unsigned long long x = pool[q * 32 + lane];
      const uint32_t mask = __ballot_sync(0xffffffffu, h[q] >= lo);
      if (h[q] >= lo) pool[c + __popc(mask & ((1u << lane) - 1u))] = x;
      c += __popc(mask);
      __syncwarp();
    }
  }
  for (int i = c + lane; i < kShortPool; i += 32) pool[i] = 0ull;
  if (sum) {
    const DoubleWeight f(m, a.iT, tab);
    double s = 0.0;
#pragma unroll 1
    for (int i = lane; i < n * kWarps; i += 32) {
      const WarpPart p = parts[i];
      if (p.m > -INFINITY) s += double(p.s) * f(p.m);
    }
    *sum = warp_sum_f64(s);
  }
  __syncwarp();
  warp_sort_pool(pool);
  return true;
}

template <typename T>
__device__ __forceinline__ bool finish_short(const TopJob& j, const RowAsk& a,
                                             const RowView<T>& rv, int row,
                                             unsigned long long* pool, double* w,
                                             const double* tab) {
  const int lane = threadIdx.x & 31;
  float m;
  double s;
  if (!short_pool(j, a, row, pool, tab, &m, j.lse ? &s : nullptr)) return false;
  if (lane == 0) j.t.left[row] = RowLeft{0, 0.0f, 0u, 0u};
  if (j.lse) {
    if (!sum_stands(j, s, m, a.iT, tab, pool, j.k))
      s = warp_sum_f64(exact_share(j.t, rv, row, m, a.iT, tab, j.c, pool, j.k, j.k, s, 0, 1));
    if (lane == 0) write_lse(j, row, m, a.iT, s);
  }
  for (int i = lane; i < j.k; i += 32) write_top(j, row, i, true, pool[i]);
  return true;
}

template <typename T>
__device__ __forceinline__ bool finish_short(const SampleJob& j, const RowAsk& a,
                                             const RowView<T>&, int row,
                                             unsigned long long* pool, double* w,
                                             const double* tab) {
  const int lane = threadIdx.x & 31;
  float m;
  if (a.bad || a.greedy || !short_pool(j, a, row, pool, tab, &m, nullptr)) return false;
  const DoubleWeight f(m, a.iT, tab);
  // the kept prefix, as kept_prefix takes it
  constexpr int kPer = kShortK / 32;
  double own = 0.0, total;
#pragma unroll 1
  for (int r = 0; r < kPer; ++r) {
    const int i = lane * kPer + r;
    const double x = i < a.K ? f(pool_value(pool[i])) : 0.0;
    w[i] = x;
    own += x;
  }
  double cum = warp_exclusive_scan(own, &total);
  const double reach = a.p * total;
  int nk = a.K;
#pragma unroll 1
  for (int r = 0; r < kPer; ++r) {
    const int i = lane * kPer + r;
    const double x = w[i];
    cum += x;
    if (i < nk && ((a.p < 1.0 && cum >= reach) || !(x > 0.0) || x < a.q))
      nk = (x > 0.0 && x >= a.q) ? i + 1 : i;
  }
  nk = max(__reduce_min_sync(0xffffffffu, nk), 1);
  // in ascending order of the ids, each with its place in w_
  __syncwarp();
  for (int i = lane; i < kShortPool; i += 32)
    pool[i] = i < nk ? (pool[i] << 32) | (unsigned long long)i : 0ull;  // (the low word is ~id)
  __syncwarp();
  warp_sort_pool(pool);
  own = 0.0;
#pragma unroll 1
  for (int r = 0; r < kPer; ++r) {
    const int i = lane * kPer + r;
    own += i < nk ? w[uint32_t(pool[i])] : 0.0;
  }
  cum = warp_exclusive_scan(own, &total);
  const double target = double(j.uniforms[row]) * total;
  int at = nk - 1;
#pragma unroll 1
  for (int r = 0; r < kPer; ++r) {
    const int i = lane * kPer + r;
    cum += i < nk ? w[uint32_t(pool[i])] : 0.0;
    if (cum > target) at = min(at, i);
  }
  at = __reduce_min_sync(0xffffffffu, at);
  if (lane == 0) {
    const unsigned long long e = pool[at];
    j.t.left[row] = RowLeft{0, 0.0f, 0u, 0u};
    write_draw(j, row, int(0xFFFFFFFFu - uint32_t(e >> 32)), w[uint32_t(e)], total);
  }
  return true;
}

template <typename T>
__device__ void finish_row(const SampleJob& j, const RowAsk& a, const RowView<T>& rv, int row,
                           PoolSmem& sm) {
  const int tid = threadIdx.x;
  if (tid == 0) j.t.left[row] = RowLeft{0, 0.0f, 0u, 0u};
  if (a.bad) {
    if (tid == 0) write_draw(j, row, -1, 0.0, 1.0);
    return;
  }
  merge_parts(j, a, row, sm);
  const float m = sm.m;
  if (sm.bad) {
    if (tid == 0) write_draw(j, row, -1, 0.0, 1.0);
    return;
  }
  if (a.greedy) {
    const WarpPart* parts = j.t.parts + size_t(row) * j.t.n * kWarps;
    for (int i = tid; i < j.t.n * kWarps; i += kThreads)
      if (parts[i].m == m) atomicMin(&sm.best, parts[i].cnt);
    __syncthreads();
    if (tid == 0) write_draw(j, row, sm.best, 1.0, 1.0);
    return;
  }
  if (a.j == 0) {
    plain_draw<T>(j, a, rv, row, sm);
    return;
  }
  if (a.j < 0 || sm.over) {
    if (tid == 0) leave_row(j.t, row, m);
    return;
  }
  const DoubleWeight f(m, a.iT, sm.tab);
  double Z = 0.0, off = 0.0;
  const float floor = a.q > 0.0 ? value_up<T>(min_p_floor(a, m)) : -INFINITY;
  float bound = sm.tau;
  int c = gather_pool(j.t, row, bound, sm, a.iT, a.sum ? &Z : nullptr);
  if (a.sum) {
    // (the lists' order is not fixed: the sum may differ in its last places, far below `off`)
    Z = block_sum_f64(Z, sm.scr) + sm.s;
    off = sum_error(j.t.V, sm.s) * sm.s + 1e-11 * (1.0 + Z);
  }
  int nk = -1;
  if (c >= 0) {
    pool_sort<true>(sm, c, a.K);
    nk = kept_prefix(a, j.t.V, c, bound, floor, Z, off, sm);
  }
  if (nk == 0 && a.K < j.t.V) {
    // The K-th of all listed entries is no larger than the row's K-th: the row has to be complete
    // from there on. (A nucleus that the pool does not hold is the deep kernel's.)
    __syncthreads();
    if (tid == 0) sm.n = 0;
    __syncthreads();
    c = gather_pool(j.t, row, -INFINITY, sm, a.iT, nullptr);
    nk = -1;
    if (c >= a.K) {
      pool_sort<true>(sm, c, a.K);
      bound = pool_value(sm.e()[a.K - 1]);
      __syncthreads();
      if (tid == 0) sm.n = 0;
      __syncthreads();
      c = gather_pool(j.t, row, bound, sm, a.iT, nullptr);
      if (c >= 0) c = complete_pool(j.t, rv, row, bound, sm);
      if (c >= 0) {
        pool_sort<true>(sm, c, a.K);
        nk = kept_prefix(a, j.t.V, c, bound, floor, 0.0, 0.0, sm);
      }
    }
  }
  if (nk <= 0) {
    if (tid == 0) {
      if (nk < 0 && a.sum && c >= 0 && sm.hi < uint32_t(c))
        leave_row(j.t, row, m, uint32_t(sm.e()[sm.hi] >> 32), uint32_t(sm.e()[sm.lo] >> 32));
      else
        leave_row(j.t, row, m);
    }
    return;
  }
  // the draw walks the kept ids in ascending order
  const double u = double(j.uniforms[row]);
  __syncthreads();
  if (nk <= 64) {
    // every entry's running sum straight from its fellows' ids (pairs of sums: the additions of
    // one chain wait for one another)
    const bool on = tid < nk;
    const int id = on ? pool_id(sm.e()[tid]) : INT_MAX;
    double c0 = 0.0, c1 = 0.0, s0 = 0.0, s1 = 0.0;
    int after = 0;
    if (warp_of(tid) < 2) {
#pragma unroll 4
      for (int i = 0; i + 1 < nk; i += 2) {
        const double w0 = sm.w()[i], w1 = sm.w()[i + 1];
        const bool b0 = pool_id(sm.e()[i]) <= id, b1 = pool_id(sm.e()[i + 1]) <= id;
        c0 += b0 ? w0 : 0.0;
        c1 += b1 ? w1 : 0.0;
        s0 += w0;
        s1 += w1;
        after += (b0 ? 0 : 1) + (b1 ? 0 : 1);
      }
      if (nk & 1) {
        const bool b0 = pool_id(sm.e()[nk - 1]) <= id;
        c0 += b0 ? sm.w()[nk - 1] : 0.0;
        s0 += sm.w()[nk - 1];
        after += b0 ? 0 : 1;
      }
    }
    const double S = s0 + s1;
    if (on && (c0 + c1 > u * S || after == 0)) atomicMin(&sm.best, id);
    __syncthreads();
    if (on && id == sm.best) write_draw(j, row, id, sm.w()[tid], S);
    return;
  }
  // longer: sort by id, the key kept beside it, and sum in that order
  for (int i = tid; i < nk; i += kThreads) {
    const unsigned long long e = sm.e()[i];
    sm.e()[i] = ((unsigned long long)pool_id(e) << 32) | (e >> 32);
  }
  __syncthreads();
  pool_sort<false>(sm, nk, nk);
  const int per2 = (nk + kThreads - 1) / kThreads, k0 = tid * per2, k1 = min(nk, k0 + per2);
  double own = 0.0, total;
  for (int i = k0; i < k1; ++i) {
    const double w = f(f32_of_key(uint32_t(sm.e()[i] & 0xFFFFFFFFull)));
    sm.w()[i] = w;
    own += w;
  }
  double cum = block_exclusive_scan(own, sm.scr, &total);
  if (tid == 0) sm.best = nk - 1;
  __syncthreads();
  for (int i = k0; i < k1; ++i) {
    cum += sm.w()[i];
    if (cum > u * total) {
      atomicMin(&sm.best, i);
      break;
    }
  }
  __syncthreads();
  if (tid == 0) write_draw(j, row, int(sm.e()[sm.best] >> 32), sm.w()[sm.best], total);
}

template <typename T>
__device__ void finish_row(const TopJob& j, const RowAsk& a, const RowView<T>& rv, int row,
                           PoolSmem& sm) {
  const int tid = threadIdx.x;
  merge_parts(j, a, row, sm);
  const float m = sm.m;
  const double S = sm.s;
  if (tid == 0) {
    j.t.left[row] = RowLeft{0, 0.0f, 0u, 0u};
    if (j.lse) {  // (once the k largest are known, the sum may be taken again)
      if (sm.bad)
        j.lse[row] = NAN;
      else
        write_lse(j, row, m, a.iT, S);
    }
  }
  if (sm.bad) {
    for (int i = tid; i < j.k; i += kThreads) {
      j.ids[size_t(row) * j.k + i] = -1;
      j.values[size_t(row) * j.k + i] = NAN;
    }
    return;
  }
  int c = -1;
  if (!sm.over) {
    float bound = sm.tau;
    c = gather_pool(j.t, row, bound, sm, a.iT, nullptr);
    if (c >= 0) pool_sort<true>(sm, c, j.k);
    if (c >= 0 && c < j.k && bound > -INFINITY) {
      // as in drawing: the k-th of all listed entries bounds the row's k-th from below
      __syncthreads();
      if (tid == 0) sm.n = 0;
      __syncthreads();
      c = gather_pool(j.t, row, -INFINITY, sm, a.iT, nullptr);
      if (c >= j.k) {
        pool_sort<true>(sm, c, j.k);
        bound = pool_value(sm.e()[j.k - 1]);
        __syncthreads();
        if (tid == 0) sm.n = 0;
        __syncthreads();
        c = gather_pool(j.t, row, bound, sm, a.iT, nullptr);
        if (c >= 0) c = complete_pool(j.t, rv, row, bound, sm);
        if (c >= 0) pool_sort<true>(sm, c, j.k);
      } else {
        c = -1;
      }
    }
  }
  if (c < 0) {
    // (the sum goes along where a nucleus would have its keys)
    if (tid == 0)
      leave_row(j.t, row, m, uint32_t(__double2loint(S)), uint32_t(__double2hiint(S)));
    return;
  }
  for (int i = tid; i < j.k; i += kThreads) write_top(j, row, i, i < c, sm.e()[i < c ? i : 0]);
  if (j.lse && !sum_stands(j, S, m, a.iT, sm.tab, sm.e(), min(c, j.k))) {
    const double all = block_sum_f64(exact_share(j.t, rv, row, m, a.iT, sm.tab, j.c, sm.e(), c,
                                                 j.k, S, tid >> 5, kWarps), sm.scr);
    if (tid == 0) write_lse(j, row, m, a.iT, all);
  }
}

// The steps in a launch each.
template <typename T, typename Job>
__global__ void __launch_bounds__(kThreads, 5) row_tile_kernel(const __grid_constant__ Job j) {
  __shared__ TileSmem tsm;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = int(blockIdx.x / unsigned(j.t.n)), tile = int(blockIdx.x % unsigned(j.t.n));
  const RowAsk a = row_ask(j, row);
  if (a.bad) return;  // (finishing does not look at the tiles)
  row_tile<T>(j, a, RowView<T>(j.t.logits, row, j.t.stride, j.t.V), row, tile, tsm);
}
template <typename T, typename Job>
__global__ void __launch_bounds__(kThreads, 4) row_finish_kernel(const __grid_constant__ Job j) {
  PoolSmem& pool = *pool_smem(j.t.pool);
  const int row = int(blockIdx.x);
  load_exp_table(pool.tab);  // (a barrier of finish_row stands before its first use)
  const RowAsk a = row_ask(j, row);
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  finish_row<T>(j, a, RowView<T>(j.t.logits, row, j.t.stride, j.t.V), row, pool);
}
template <typename T, typename Job>
__global__ void __launch_bounds__(kThreads, 3) row_short_kernel(const __grid_constant__ Job j) {
  PoolSmem& sm = *pool_smem(j.t.pool);
  load_exp_table(sm.tab);
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
  const int row0 = int(blockIdx.x) * kWarps, warp = threadIdx.x >> 5;
  bool done = true;
  if (row0 + warp < j.t.rows) {
    unsigned long long* pool = sm.e() + warp * kShortRoom;
    double* w = reinterpret_cast<double*>(sm.e() + kWarps * kShortRoom) + warp * kShortK;
    const int row = row0 + warp;
    done = finish_short(j, row_ask(j, row), RowView<T>(j.t.logits, row, j.t.stride, j.t.V), row,
                        pool, w, sm.tab);
  }
#pragma unroll 1
  for (int q = 0; q < kWarps; ++q)
    if (__syncthreads_or(warp == q && !done)) {
      const int row = row0 + q;
      finish_row<T>(j, row_ask(j, row), RowView<T>(j.t.logits, row, j.t.stride, j.t.V), row, sm);
    }
}
inline size_t short_bytes(int cap) {
  const size_t own = sizeof(PoolSmem) + kWarps * (kShortRoom * sizeof(unsigned long long) +
                                                  kShortK * sizeof(double));
  const size_t pool = pool_bytes(cap);
  return own > pool ? own : pool;
}

// ------------------------------------------------------------------------- whole rows
// Rows that the pool does not settle: a kept set longer than the pool, a top_k that the lists do
// not aim at, thousands of equal values at a threshold, a decision within the error bound of the
// float32 sums. A cluster of kDeepCtas blocks takes a row, each an adjacent part of it (which
// stays in its SM's L1), from the list that the finishing blocks left.
//   Top-k's cut: counts of entries over 1,024 ranges of the order keys (16 or 32 bits), from the
//   largest down; the range that holds the k-th is split again until its entries can be sorted, or
//   share one key.
//   Top-p's cut, where the pool holds it but the float32 sum leaves it open between two of its
//   entries: one double pass sums the mass above these and in all, and lists what lies between (64
//   rows of 128,256, twelve inputs: 60.8 -> 56.2 us a call). Else counts over 1,024 equal steps
//   of (m - l) / T up to 46 (what lies below weighs
//   less than 1e-20 of the largest entry, 1e-14 of it in all, and does not move the cut). A step's
//   mass is its count times something between the weights at its ends, so the cut lies in a few
//   steps; one double pass sums the mass above them and in all, and they are split again, with what
//   is left of the mass as the target. (Every block reads all histograms: with 4,096 bins that alone
//   took 8 us of a search's 12.)
//   The draw: double sums of the blocks' warps' adjacent parts, then of the threads' in the part
//   that holds the target.
// Shapes and orders of all sums are fixed within a call (how many other rows are left decides whether
// a row is summed by one block or by eight); atomics only count and fill lists that are sorted.
constexpr int kDeepCtas = 8;
constexpr int kDeepThreads = 512;
constexpr int kDeepWarps = kDeepThreads / 32;
constexpr int kDeepBins = 1024;
constexpr int kDeepCap = 1024;                      // entries the first block of a cluster sorts
constexpr double kDeepNats = 46.0;

struct DeepSmem {
  uint32_t hist[kDeepBins];
  uint16_t rows[4 * kDeepThreads];
  unsigned long long e[kDeepCap];
  double tab[64];
  double red[2][2];                 // this block's partial sums, two turns
  double part[2][kDeepWarps];       // its warps' sums, two turns
  double scr[kDeepWarps], scr2[kDeepWarps];
  uint32_t scr_u[kDeepWarps];
  uint32_t kmin, kmax, n;           // the cluster's, in its first block
  uint32_t thr, cutoff;             // its decision
  uint32_t b0, b1, above, inside;   // a search's answer, in every block
  int best, last, sel;
  double base, total;
  // An entry for the first block's list (any block calls it on that block's memory).
  __device__ __forceinline__ void push(uint32_t key, int id) {
    const uint32_t at = atomicAdd(&n, 1u);
    if (at < uint32_t(kDeepCap))
      e[at] = ((unsigned long long)key << 32) | (unsigned long long)(0xFFFFFFFFu - uint32_t(id));
  }
};

// kBlock threads a block.
template <typename T, int kBlock>
struct Deep {
  static constexpr int kW = kBlock / 32;
  static constexpr int kPerBins = kDeepBins / kBlock;   // bins a thread scans
  static constexpr int kPerList = kDeepCap / kBlock;    // list entries a thread takes
  cg::cluster_group cl;
  DeepSmem& sm;
  RowView<T> rv;
  float m;
  DoubleWeight w;
  int ctas;             // blocks that share the row: the cluster's, or this one alone
  int rank, g0, g1;     // this block's vectors
  int turn = 0;
  uint32_t thr = 0u;    // kept: key > thr, or key == thr and id <= cutoff
  uint32_t cutoff = 0x7FFFFFFFu;

  __device__ Deep(DeepSmem& s, const RowView<T>& v, float m_, double iT, int ctas_)
      : cl(cg::this_cluster()), sm(s), rv(v), m(m_), w(m_, iT, s.tab), ctas(ctas_) {
    rank = ctas == 1 ? 0 : int(cl.block_rank());
    const int per = (rv.G + ctas - 1) / ctas;
    g0 = min(rv.G, rank * per);
    g1 = min(rv.G, g0 + per);
  }
  // Order-preserving key at the type's own width, and its value.
  static constexpr int kDown = 32 - Elem<T>::kKeyBits;
  __device__ static __forceinline__ uint32_t key_of(float x) { return f32_key(x) >> kDown; }
  __device__ static __forceinline__ float value_of(uint32_t k) {
    const uint32_t u = k << kDown;
    return f32_of_key((u & 0x80000000u) ? u : u | ((1u << kDown) - 1u));
  }
  __device__ __forceinline__ void sync() {
    if (ctas == 1)
      __syncthreads();
    else
      cl.sync();
  }
  __device__ __forceinline__ DeepSmem* of(int r) {
    return ctas == 1 ? &sm : cl.map_shared_rank(&sm, unsigned(r));
  }
  __device__ DeepSmem& first() { return *of(0); }
  __device__ bool in(uint32_t key, int id) const {
    return key > thr || (key == thr && uint32_t(id) <= cutoff);
  }

  // f(x, key, id) for this block's entries above -inf.
  template <typename F>
  __device__ __forceinline__ void each(F&& f) {
    constexpr int P = Elem<T>::kPerVec;
    int g = g0 + int(threadIdx.x);
    if (g >= g1) return;
    uint4 v = rv.load(g);
#pragma unroll 1
    for (; g < g1; g += kBlock) {
      const uint4 cur = v;
      if (g + kBlock < g1) v = rv.load(g + kBlock);
      float x[P];
      Elem<T>::unpack(cur, x);
      const int e0 = rv.first(g);
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (x[e] > -INFINITY) f(x[e], key_of(x[e]), e0 + e);
    }
  }

  // Sums over the cluster of two values of every thread.
  __device__ void sum2(double& a, double& b) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = warp_sum_f64(a);
    b = warp_sum_f64(b);
    __syncthreads();
    if (lane == 0) {
      sm.scr[warp] = a;
      sm.scr2[warp] = b;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      a = b = 0.0;
      for (int q = 0; q < kW; ++q) {
        a += sm.scr[q];
        b += sm.scr2[q];
      }
      sm.red[turn][0] = a;
      sm.red[turn][1] = b;
    }
    sync();
    a = b = 0.0;
#pragma unroll
    for (int r = 0; r < kDeepCtas; ++r)
      if (r < ctas) {
        const DeepSmem* o = of(r);
        a += o->red[turn][0];
        b += o->red[turn][1];
      }
    turn ^= 1;
  }

  __device__ void clear_hist() {
    for (int i = threadIdx.x; i < kDeepBins; i += kBlock) sm.hist[i] = 0u;
    if (threadIdx.x == 0) {
      sm.n = 0u;
      sm.kmin = 0xFFFFFFFFu;
      sm.kmax = 0u;
    }
    __syncthreads();
  }

  // After the blocks have counted into their histograms (bin 0 holds the largest values): the
  // bins where the running count reaches k (kMass false), or from the first where the running
  // mass can reach the target to the first where it must have (kMass true). lo(b) and hi(b)
  // bound an entry's weight in bin b; the target is t, or t times the bins' whole mass when
  // rel. Answers in sm.b0, b1, above (entries before b0) and inside (entries of b0..b1), in
  // every block alike. k = 0 asks for the last entry there is. Ends with the histograms free.
  template <bool kMass, typename Lo, typename Hi>
  __device__ void search(uint32_t k, bool rel, double t, Lo&& lo, Hi&& hi) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    sync();
    uint32_t c[kPerBins];
    double l[kPerBins], h[kPerBins];  // the bins' masses at the least and the most
#pragma unroll
    for (int q = 0; q < kPerBins; ++q) {
      c[q] = 0u;
      l[q] = h[q] = 0.0;
    }
#pragma unroll
    for (int r = 0; r < kDeepCtas; ++r)
      if (r < ctas) {
        const uint32_t* from = of(r)->hist + tid * kPerBins;
#pragma unroll
        for (int q = 0; q < kPerBins; ++q) c[q] += from[q];
      }
    uint32_t own = 0u;
    double lo_own = 0.0, hi_own = 0.0;
#pragma unroll
    for (int q = 0; q < kPerBins; ++q) {
      own += c[q];
      if (kMass && c[q]) {
        l[q] = double(c[q]) * lo(uint32_t(tid * kPerBins + q));
        h[q] = double(c[q]) * hi(uint32_t(tid * kPerBins + q));
        lo_own += l[q];
        hi_own += h[q];
      }
    }
    uint32_t inc = own;
    double li = lo_own, hx = hi_own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
      if (kMass) {
        const double a = __shfl_up_sync(0xffffffffu, li, o), b = __shfl_up_sync(0xffffffffu, hx, o);
        if (lane >= o) {
          li += a;
          hx += b;
        }
      }
    }
    if (lane == 31) {
      sm.scr_u[warp] = inc;
      sm.scr[warp] = li;
      sm.scr2[warp] = hx;
    }
    if (tid == 0) sm.b0 = sm.b1 = 0xFFFFFFFFu;
    __syncthreads();
    uint32_t n = inc - own, all = 0u;
    double ml = li - lo_own, mh = hx - hi_own, zl = 0.0, zh = 0.0;
    for (int q = 0; q < kW; ++q) {
      if (q < warp) {
        n += sm.scr_u[q];
        if (kMass) {
          ml += sm.scr[q];
          mh += sm.scr2[q];
        }
      }
      all += sm.scr_u[q];
      if (kMass) {
        zl += sm.scr[q];
        zh += sm.scr2[q];
      }
    }
    const uint32_t kk = k == 0u ? all : min(k, all);
    // (running sums in another order differ in the last places: 1e-12 to each side)
    const double tl = (rel ? t * zl : t) * (1.0 - 1e-12), th = (rel ? t * zh : t) * (1.0 + 1e-12);
#pragma unroll
    for (int q = 0; q < kPerBins; ++q) {
      if (c[q] == 0u) continue;
      const uint32_t b = uint32_t(tid * kPerBins + q);
      n += c[q];
      if (kMass) {
        ml += l[q];
        mh += h[q];
        if (mh >= tl) atomicMin(&sm.b0, b);
        if (ml >= th || n == all) atomicMin(&sm.b1, b);
      } else if (n >= kk) {
        atomicMin(&sm.b0, b);
        atomicMin(&sm.b1, b);
      }
    }
    __syncthreads();
    const uint32_t b1 = sm.b1, b0 = min(sm.b0, b1);
    __syncthreads();
    // counts up to the two bins
    uint32_t before = inc - own;
    for (int q = 0; q < warp; ++q) before += sm.scr_u[q];
#pragma unroll
    for (int q = 0; q < kPerBins; ++q) {
      const uint32_t b = uint32_t(tid * kPerBins + q);
      if (b == b0) sm.above = before;
      before += c[q];
      if (b == b1) sm.inside = before;
    }
    if (tid == 0) sm.b0 = b0;
    __syncthreads();
    if (tid == 0) sm.inside -= sm.above;
    sync();
  }

  // The entry id at which the running sum over the ids of f(x, key, id) >= 0 (entries above
  // -inf) passes target(total); the last with f > 0 where rounding leaves none. Every block
  // returns it; *total gets the sum.
  template <typename F, typename G>
  __device__ int locate(F&& f, G&& target, double* total) {
    constexpr int P = Elem<T>::kPerVec;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int span = (g1 - g0 + kW - 1) / kW;
    const int w0 = min(g1, g0 + warp * span), w1 = min(g1, w0 + span);
    double s = 0.0;
    uint4 v = w0 + lane < w1 ? rv.load(w0 + lane) : neg_inf_vec(int(sizeof(T)));
#pragma unroll 1
    for (int g = w0 + lane; g < w1; g += 32) {
      const uint4 cur = v;
      if (g + 32 < w1) v = rv.load(g + 32);
      float x[P];
      Elem<T>::unpack(cur, x);
      const int e0 = rv.first(g);
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (x[e] > -INFINITY) s += f(x[e], key_of(x[e]), e0 + e);
    }
    s = warp_sum_f64(s);
    if (lane == 0) sm.part[turn][warp] = s;
    if (tid == 0) {
      sm.best = INT_MAX;
      sm.last = -1;
    }
    sync();
    if (warp == 0) {
      // adjacent parts to a lane
      constexpr int kPer = kDeepCtas * kW / 32;
      const int r = lane * kPer / kW;
      double p[kPer], own = 0.0;
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        p[q] = r < ctas ? of(r)->part[turn][lane * kPer % kW + q] : 0.0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) own += p[q];
      double inc = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += up;
      }
      const double S = __shfl_sync(0xffffffffu, inc, 31);
      const double t = target(S);
      double cum = inc - own, before = 0.0, last_before = 0.0;
      int sel = -1, last = -1;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (p[q] > 0.0) {
          last = lane * kPer + q;
          last_before = cum;
          if (sel < 0 && cum + p[q] > t) {
            sel = last;
            before = cum;
          }
        }
        cum += p[q];
      }
      // the first part that passes the target, else the last with mass
      const uint32_t hit = __ballot_sync(0xffffffffu, sel >= 0);
      const uint32_t any = __ballot_sync(0xffffffffu, last >= 0);
      const int from = hit ? __ffs(int(hit)) - 1 : (any ? 31 - __clz(int(any)) : 0);
      if (lane == from) {
        sm.sel = hit ? sel : max(last, 0);
        sm.base = hit ? before : last_before;
        sm.total = S;
      }
    }
    turn ^= 1;
    __syncthreads();
    *total = sm.total;
    const int owner = sm.sel / kW;
    if (owner == rank) {
      const double t = target(sm.total);
      const int r0 = min(g1, g0 + (sm.sel % kW) * span), r1 = min(g1, r0 + span);
      const int per = (span + kBlock - 1) / kBlock;
      const int a0 = min(r1, r0 + tid * per), a1 = min(r1, a0 + per);
      double own = 0.0, q0[P];  // (the weights of the thread's first vector, often its only one)
      int last = -1;
#pragma unroll
      for (int e = 0; e < P; ++e) q0[e] = 0.0;
#pragma unroll 1
      for (int g = a0; g < a1; ++g) {
        float x[P];
        Elem<T>::unpack(rv.load(g), x);
        const int e0 = rv.first(g);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const double q = x[e] > -INFINITY ? f(x[e], key_of(x[e]), e0 + e) : 0.0;
          if (g == a0) q0[e] = q;
          own += q;
          if (q > 0.0) last = e0 + e;
        }
      }
      double inc = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) sm.scr[warp] = inc;
      __syncthreads();
      double cum = sm.base;
      for (int q = 0; q < warp; ++q) cum += sm.scr[q];
      cum += inc - own;
      if (last >= 0) {
        atomicMax(&sm.last, last);
        if (cum + own > t) {
          bool found = false;
          const int e0 = rv.first(a0);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            cum += q0[e];
            if (!found && q0[e] > 0.0 && cum > t) {
              atomicMin(&sm.best, e0 + e);
              found = true;
            }
          }
#pragma unroll 1
          for (int g = a0 + 1; g < a1 && !found; ++g) {
            float x[P];
            Elem<T>::unpack(rv.load(g), x);
            const int e1 = rv.first(g);
            for (int e = 0; e < P && !found; ++e)
              if (x[e] > -INFINITY) {
                const double q = f(x[e], key_of(x[e]), e1 + e);
                cum += q;
                if (q > 0.0 && cum > t) {
                  atomicMin(&sm.best, e1 + e);
                  found = true;
                }
              }
          }
        }
      }
      __syncthreads();
      if (tid == 0 && sm.best == INT_MAX) sm.best = sm.last;
    }
    sync();
    const int id = of(owner)->best;
    sync();
    return id;
  }

  // Sets the cut at the entry, among the listed `inside` ones or (one key, more than the list takes)
  // those with key kmax that are in the kept set so far, where the count reaches k or the mass from
  // A on reaches P.
  template <bool kMass>
  __device__ void cut_at(uint32_t kmax, uint32_t inside, uint32_t k, double A, double P) {
    DeepSmem& d = first();
    if (inside <= uint32_t(kDeepCap)) {
      if (rank == 0) {
        const int n = min(int(sm.n), kDeepCap), N = pow2_at_least(n);
        for (int i = n + int(threadIdx.x); i < N; i += kBlock) sm.e[i] = 0ull;
        __syncthreads();
        block_sort<true, kBlock>(sm.e, N);
        int at = min(n - 1, int(k) - 1);
        if (kMass) {
          // the first entry whose running mass reaches P
          const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
          double we[kPerList], own = 0.0;
#pragma unroll
          for (int e = 0; e < kPerList; ++e) {
            const int i = tid * kPerList + e;
            we[e] = i < n ? w(value_of(uint32_t(sm.e[i] >> 32))) : 0.0;
            own += we[e];
          }
          double inc = own;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
          }
          if (lane == 31) sm.scr[warp] = inc;
          if (tid == 0) sm.best = n - 1;
          __syncthreads();
          double cum = A;
          for (int q = 0; q < warp; ++q) cum += sm.scr[q];
          cum += inc - own;
#pragma unroll
          for (int e = 0; e < kPerList; ++e) {
            cum += we[e];
            if (tid * kPerList + e < n && cum >= P) {
              atomicMin(&sm.best, tid * kPerList + e);
              break;
            }
          }
          __syncthreads();
          at = sm.best;
        }
        if (threadIdx.x == 0) {
          sm.thr = uint32_t(sm.e[at] >> 32);
          sm.cutoff = uint32_t(pool_id(sm.e[at]));
        }
      }
      sync();
      thr = d.thr;
      cutoff = d.cutoff;
      sync();
      return;
    }
    double r = double(k), n;
    if (kMass) {
      const double w0 = w(value_of(kmax));
      r = w0 > 0.0 ? fmin(fmax(ceil((P - A) / w0), 1.0), double(inside)) : 1.0;
    }
    const int id = locate([&](float, uint32_t key, int i) { return key == kmax && in(key, i) ? 1.0 : 0.0; },
                          [&](double) { return r - 0.5; }, &n);
    thr = kmax;
    cutoff = uint32_t(id);
  }

  // Keeps the k largest entries (all above -inf when there are fewer): the keys' range that holds
  // the k-th is split until its entries fit the list or share one key.
  __device__ void cut_top_k(uint32_t k) {
    uint32_t kmin = 0x00800000u >> kDown, kmax = key_of(m), above = 0u, inside = uint32_t(rv.V);
    while (inside > uint32_t(kDeepCap) && kmin < kmax) {
      const int bits = 32 - __clz(int(kmax - kmin));
      const int sh = bits > 10 ? bits - 10 : 0;
      clear_hist();
      each([&](float, uint32_t key, int) {
        if (key >= kmin && key <= kmax) atomicAdd(&sm.hist[(kmax - key) >> sh], 1u);
      });
      search<false>(k - above, false, 0.0, [](uint32_t) { return 0.0; },
                    [](uint32_t) { return 0.0; });
      const uint32_t step = (1u << sh) - 1u, range = kmax - kmin, b = sm.b0 << sh;
      above += sm.above;
      inside = sm.inside;
      kmin = kmax - min(range, b + step);
      kmax = kmax - b;
      __syncthreads();
    }
    if (inside <= uint32_t(kDeepCap)) {
      if (threadIdx.x == 0) sm.n = 0u;
      sync();
      DeepSmem& d = first();
      each([&](float, uint32_t key, int id) {
        if (key >= kmin && key <= kmax) d.push(key, id);
      });
      sync();
    }
    cut_at<false>(kmax, inside, k - above, 0.0, 0.0);
  }

  // Of the kept entries, keeps the shortest prefix whose mass reaches p of theirs. Each level cuts
  // the values that may hold the crossing into equal steps (in keys, whose steps grow with the
  // value's distance from 0, a step's ends may weigh 50 times as much as one another), narrows them
  // down, and sums what lies above in double.
  // Where lo > 0, the cut is known to lie among the keys from lo to hi (of 32 bits).
  __device__ void cut_top_p(double p, double iT, uint32_t lo32, uint32_t hi32) {
    const double h = kDeepNats / kDeepBins;
    float top = m;                                       // bin 0 begins here
    float s = float(fmin(iT / h, 1e37));                 // bins per unit of value
    uint32_t lo = 0u, hi = 0xFFFFFFFFu, inside = 0u;     // keys that may hold the crossing
    double A = 0.0, Z = 0.0, P = 0.0;
    bool listed = false;
    const bool known = lo32 > 0u;
    if (known) {
      lo = lo32 >> kDown;
      hi = hi32 >> kDown;
      if (threadIdx.x == 0) sm.n = 0u;
      sync();
      DeepSmem& d = first();
      each([&](float x, uint32_t key, int id) {
        const double q = w(x);
        Z += q;
        if (key > hi) A += q;
        if (key >= lo && key <= hi) d.push(key, id);
      });
      sum2(A, Z);
      P = p * Z;
      inside = d.n;
      listed = inside <= uint32_t(kDeepCap);
      sync();
    }
    for (int level = known ? 1 : 0; level == 0 || (inside > uint32_t(kDeepCap) && lo < hi); ++level) {
      if (level) {
        top = value_of(hi);
        s = float(kDeepBins - 1) / (top - value_of(lo));
      }
      auto bin = [&](float x) {
        const int b = __float2int_rz((top - x) * s);
        return level ? min(b, kDeepBins - 1) : b;
      };
      clear_hist();
      each([&](float x, uint32_t key, int id) {
        if (key < lo || key > hi) return;
        const int b = bin(x);
        if (b < kDeepBins && in(key, id)) atomicAdd(&sm.hist[b], 1u);
      });
      // an entry of bin b lies b / s to (b + 1) / s below top, but for the float roundings of the
      // difference, of s and of their product
      const double off = (double(m) - double(top)) * iT, per = iT / double(s);
      search<true>(0u, level == 0, level == 0 ? p : P - A,
                   [&](uint32_t b) { return exp_neg(-(off + (double(b) + 1.0) * per * (1.0 + 1e-6))); },
                   [&](uint32_t b) { return exp_neg(-(off + double(b) * per * (1.0 - 1e-6))); });
      const int b0 = int(sm.b0), b1 = int(sm.b1);
      DeepSmem& d = first();
      double a = 0.0, z = 0.0;
      uint32_t kmin = 0xFFFFFFFFu, kmax = 0u;
      if (level && sm.inside == inside) {
        // Nothing was ruled out: the first step holds about what is wanted, and what follows little.
        // Its exact mass tells on which side the crossing lies.
        double in_first = 0.0;
        uint32_t rest = 0u;
        each([&](float x, uint32_t key, int id) {
          if (key < lo || key > hi || !in(key, id)) return;
          if (bin(x) == 0) {
            a += w(x);
            in_first += 1.0;
            kmin = min(kmin, key);
          } else {
            rest = max(rest, key);
          }
        });
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        rest = __reduce_max_sync(0xffffffffu, rest);
        if ((threadIdx.x & 31) == 0) {
          atomicMin(&d.kmin, kmin);
          atomicMax(&d.kmax, rest);
        }
        sum2(a, in_first);
        if (A + a >= P) {
          lo = d.kmin;
          inside = uint32_t(in_first);
        } else {
          hi = d.kmax;
          A += a;
          inside -= uint32_t(in_first);
        }
        sync();
        listed = false;
        continue;
      }
      inside = sm.inside;
      const bool take = inside <= uint32_t(kDeepCap);
      listed = take;
      each([&](float x, uint32_t key, int id) {
        if (key < lo || key > hi || !in(key, id)) return;
        const int b = bin(x);
        if (level && b > b1) return;
        if (level == 0 || b < b0) {
          const double q = w(x);
          z += q;
          if (b < b0) a += q;
        }
        if (b >= b0 && b <= b1) {
          kmin = min(kmin, key);
          kmax = max(kmax, key);
          if (take) d.push(key, id);
        }
      });
      kmin = __reduce_min_sync(0xffffffffu, kmin);
      kmax = __reduce_max_sync(0xffffffffu, kmax);
      if ((threadIdx.x & 31) == 0) {
        atomicMin(&d.kmin, kmin);
        atomicMax(&d.kmax, kmax);
      }
      sum2(a, z);
      lo = d.kmin;
      hi = d.kmax;
      sync();
      A += a;
      if (level == 0) {
        Z = z;
        P = p * Z;
      }
    }
    if (!listed && inside <= uint32_t(kDeepCap)) {
      if (threadIdx.x == 0) sm.n = 0u;
      sync();
      DeepSmem& d = first();
      each([&](float, uint32_t key, int id) {
        if (key >= lo && key <= hi && in(key, id)) d.push(key, id);
      });
      sync();
    }
    cut_at<true>(hi, inside, 0u, A, P);
  }
};

// A whole row by `ctas` blocks of kBlock threads.
template <typename T, int kBlock>
__device__ void deep_row(const SampleJob& j, int row, const RowLeft& left, int ctas, DeepSmem& sm) {
  const RowAsk a = row_ask(j, row);
  const float m = left.m;
  Deep<T, kBlock> d(sm, RowView<T>(j.t.logits, row, j.t.stride, j.t.V), m, a.iT, ctas);
  if (a.K < j.t.V) d.cut_top_k(uint32_t(a.K));
  if (a.p < 1.0) d.cut_top_p(a.p, a.iT, left.lo, left.hi);
  double S;
  const double u = double(j.uniforms[row]);
  const float floor = a.q > 0.0 ? min_p_floor(a, m) : -INFINITY;
  const int tok = d.locate(
      [&](float x, uint32_t key, int id) {
        if (x < floor || !d.in(key, id)) return 0.0;
        const double w = d.w(x);
        return w >= a.q ? w : 0.0;
      },
      [&](double total) { return u * total; }, &S);
  if (d.rank == 0 && threadIdx.x == 0) write_draw(j, row, tok, d.w(d.rv.entry(tok)), S);
}

template <typename T, int kBlock>
__device__ void deep_row(const TopJob& j, int row, const RowLeft& left, int ctas, DeepSmem& sm) {
  const float m = left.m;
  const double iT = 1.0 / double(j.temp);
  Deep<T, kBlock> d(sm, RowView<T>(j.t.logits, row, j.t.stride, j.t.V), m, iT, ctas);
  d.cut_top_k(uint32_t(j.k));
  if (threadIdx.x == 0) sm.n = 0u;
  d.sync();
  DeepSmem& f = d.first();
  d.each([&](float x, uint32_t key, int id) {
    if (d.in(key, id)) f.push(f32_key(x), id);
  });
  d.sync();
  if (d.rank == 0) {
    const int n = min(int(sm.n), kDeepCap), N = pow2_at_least(n);
    for (int q = n + int(threadIdx.x); q < N; q += kBlock) sm.e[q] = 0ull;
    __syncthreads();
    block_sort<true, kBlock>(sm.e, N);
    for (int q = threadIdx.x; q < j.k; q += kBlock)
      write_top(j, row, q, q < n, sm.e[q < n ? q : 0]);
    const double S = __hiloint2double(int(left.hi), int(left.lo));
    if (j.lse && !sum_stands(j, S, m, iT, sm.tab, sm.e, min(n, j.k))) {
      const int warp = threadIdx.x >> 5;
      const double own = warp_sum_f64(exact_share(j.t, d.rv, row, m, iT, sm.tab, j.c, sm.e, n, j.k,
                                                  S, warp, kBlock / 32));
      if ((threadIdx.x & 31) == 0) sm.scr[warp] = own;
      __syncthreads();
      double all = 0.0;
      for (int q = 0; q < kBlock / 32; ++q) all += sm.scr[q];
      if (threadIdx.x == 0) write_lse(j, row, m, iT, all);
    }
  }
  d.sync();
}

// Calls f(row, m, ctas) for this cluster's share of the rows left: the i-th of them is cluster
// i mod clusters'. The flags are read 2,048 rows at a time by every block, which agree on the order.
// A row takes a cluster about 40 us + V / 4 ns and a block alone 25 us + 2.2 V ns (measured at V of
// 8,753 to 151,936): where so many are left that blocks by themselves are done sooner, each takes
// a row of its own (123 rows of 102,647: 543 -> 300 us).
template <typename F>
__device__ void for_rows_left(const TileJob& t, DeepSmem& sm, F&& f) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int clusters = int(gridDim.x) / kDeepCtas, mine = int(blockIdx.x) / kDeepCtas;
  constexpr int kPer = 4;
  int seen = 0;
#pragma unroll 1
  for (int r0 = 0; r0 < t.rows; r0 += kPer * kDeepThreads) {
    uint32_t todo = 0u;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int r = r0 + tid * kPer + q;
      if (r < t.rows && t.left[r].todo) todo |= 1u << q;
    }
    if (!__syncthreads_or(todo != 0u)) continue;
    int inc = __popc(todo);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) sm.scr_u[warp] = uint32_t(inc);
    __syncthreads();
    int at = inc - __popc(todo), all = 0;
    for (int q = 0; q < kDeepWarps; ++q) {
      if (q < warp) at += int(sm.scr_u[q]);
      all += int(sm.scr_u[q]);
    }
    // the chunk's rows in order
    uint16_t* rows = sm.rows;
    for (int q = 0; q < kPer; ++q)
      if (todo >> q & 1u) rows[at++] = uint16_t(tid * kPer + q);
    __syncthreads();
    const long long by_cluster = (long long)((all + clusters - 1) / clusters) * (40000 + t.V / 4);
    const long long alone =
        (long long)((all + int(gridDim.x) - 1) / int(gridDim.x)) * (25000 + t.V * 11LL / 5);
    const bool solo = alone < by_cluster;
    const int step = solo ? int(gridDim.x) : clusters;
    const int first = solo ? int(blockIdx.x) : ((mine - seen) % clusters + clusters) % clusters;
    for (int i = first; i < all; i += step) {
      const int r = r0 + int(rows[i]);
      f(r, t.left[r], solo ? 1 : kDeepCtas);
    }
    seen += all;
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kDeepThreads, 1) sample_deep_kernel(const SampleJob j) {
  __shared__ DeepSmem sm;
  load_exp_table(sm.tab);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for_rows_left(j.t, sm, [&](int row, const RowLeft& left, int ctas) {
    deep_row<T, kDeepThreads>(j, row, left, ctas, sm);
  });
}

template <typename T>
__global__ void __launch_bounds__(kDeepThreads, 1) top_deep_kernel(const TopJob j) {
  __shared__ DeepSmem sm;
  load_exp_table(sm.tab);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for_rows_left(j.t, sm, [&](int row, const RowLeft& left, int ctas) {
    deep_row<T, kDeepThreads>(j, row, left, ctas, sm);
  });
}

// Everything in one launch, for calls whose blocks are on the GPU at once: a row by a cluster of
// `blocks` blocks, the tiles first; then its first block finishes it, and where its pool does not
// settle it, the cluster goes over the whole row.
template <typename T, typename Job>
__global__ void __launch_bounds__(kThreads, 2) row_kernel(const __grid_constant__ Job j) {
  extern __shared__ __align__(16) unsigned char sv_pool[];
  TileSmem& tsm = *reinterpret_cast<TileSmem*>(sv_pool);  // then the pool, then DeepSmem
  const int row = int(blockIdx.x) / j.t.blocks, rank = int(blockIdx.x) % j.t.blocks;
  const RowAsk a = row_ask(j, row);
  const RowView<T> rv(j.t.logits, row, j.t.stride, j.t.V);
  if (!a.bad)
    for (int tile = rank; tile < j.t.n; tile += j.t.blocks) {
      if (tile != rank) __syncthreads();
      row_tile<T>(j, a, rv, row, tile, tsm);
    }
  cg::this_cluster().sync();
  if (rank == 0) {
    PoolSmem& pool = *pool_smem(j.t.pool);
    load_exp_table(pool.tab);  // (a barrier of finish_row stands before its first use)
    finish_row<T>(j, a, rv, row, pool);
  }
  cg::this_cluster().sync();
  const RowLeft left = j.t.left[row];
  if (!left.todo) return;
  DeepSmem& sm = *reinterpret_cast<DeepSmem*>(sv_pool);
  load_exp_table(sm.tab);
  __syncthreads();
  deep_row<T, kThreads>(j, row, left, j.t.blocks, sm);
  cg::this_cluster().sync();
}

}  // namespace sv

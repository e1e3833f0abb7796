// Logit rows cut into tiles: the part that drawing (sample.cuh), the top logits of a row
// (sample.cuh) and the distillation loss (distill.cuh) share.
//
// A row is seen as 16-byte vectors of the address space: vector g holds entries
// [g P - mis, g P - mis + P), P entries to a vector and mis the row's distance, in entries, from
// the 16-byte boundary below it. Full vectors are loaded whole; the ragged ones at the row's two
// ends entry by entry, with -inf outside the row, so any row address and stride of whole
// entries is read without touching its neighbours.
//
// A tile is kTileVecs vectors for each of a block's kThreads threads, in pieces of 32 adjacent
// vectors (512 bytes, a warp's load). One block takes one tile, whatever the number of rows: a
// single row of 128,256 bfloat16 entries is spread over 8 blocks, and of many rows four to six
// blocks share an SM, so that one's loads fly while another computes (2,048 x 32,000, the loss's
// sums: 27 us, 4.8 TB/s). Contiguous tiles keep the
// order of the ids, which a draw's running sum needs. Interleaved tiles, which take the row's
// pieces in turn, are samples of the whole row: vocabularies are ordered by frequency, so
// contiguous tiles would differ widely in how many of the largest entries they hold.
#pragma once

#include "draw.cuh"

namespace sv {

constexpr int kTileVecs = 8;
constexpr int kTileVectors = kTileVecs * kThreads;  // 16-byte vectors of a tile
constexpr int kMaxTiles = 129;                      // 2^20 float32 entries, a vector more if off

// kOnce = false: the row may be written by this kernel (after it has been read).
template <typename T, bool kOnce = true>
struct RowView {
  const T* row;
  int V;
  int mis;  // entries between the 16-byte boundary below the row and the row
  int G;    // vectors
  __device__ __forceinline__ RowView(const void* base, long long row_idx, long long stride, int V_)
      : row(static_cast<const T*>(base) + row_idx * stride), V(V_) {
    mis = int((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    G = (V + mis + Elem<T>::kPerVec - 1) / Elem<T>::kPerVec;
  }
  __device__ __forceinline__ int first(int g) const { return g * Elem<T>::kPerVec - mis; }
  __device__ __forceinline__ bool whole(int g) const {
    const int e = first(g);
    return e >= 0 && e + Elem<T>::kPerVec <= V;
  }
  template <typename U>
  __device__ __forceinline__ static U get(const U* p) {
    if constexpr (kOnce)
      return __ldg(p);
    else
      return *p;
  }
  __device__ __forceinline__ float entry(int id) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(get(reinterpret_cast<const uint32_t*>(row) + id));
    else
      return __uint_as_float(uint32_t(get(reinterpret_cast<const unsigned short*>(row) + id)) << 16);
  }
  // Vector g (g < G): -inf outside the row.
  __device__ __forceinline__ uint4 load(int g) const {
    const int e = first(g);
    if (e >= 0 && e + Elem<T>::kPerVec <= V) return get(reinterpret_cast<const uint4*>(row + e));
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (sizeof(T) == 4) {
        const int i = e + q;
        w[q] = (i >= 0 && i < V) ? get(reinterpret_cast<const uint32_t*>(row) + i) : 0xFF800000u;
      } else {
        const int i = e + 2 * q;
        const uint32_t lo = (i >= 0 && i < V)
                                ? get(reinterpret_cast<const unsigned short*>(row) + i) : 0xFF80u;
        const uint32_t hi = (i + 1 >= 0 && i + 1 < V)
                                ? get(reinterpret_cast<const unsigned short*>(row) + i + 1)
                                : 0xFF80u;
        w[q] = lo | (hi << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ uint4 neg_inf_vec(int elem_bytes) {
  const uint32_t w = elem_bytes == 4 ? 0xFF800000u : 0xFF80FF80u;
  return make_uint4(w, w, w, w);
}

// Running maximum of a thread's vectors, NaN if any entry is: packed for bfloat16.
template <typename T>
struct VecMax;
template <>
struct VecMax<float> {
  float m;
  __device__ __forceinline__ void add(const uint4& w, bool first) {
    const float v = Elem<float>::vmax_nan(w);
    m = first ? v : fmax_nan(m, v);
  }
  __device__ __forceinline__ void join(const VecMax& o, bool first) {
    m = first ? o.m : fmax_nan(m, o.m);
  }
  __device__ __forceinline__ float value() const { return m; }
  // Whether an entry above -inf reaches tau.
  __device__ __forceinline__ bool reaches(float tau) const { return m >= tau && m > -INFINITY; }
};
template <>
struct VecMax<__nv_bfloat16> {
  __nv_bfloat162 m;
  __device__ __forceinline__ void add(const uint4& w, bool first) {
    using E = Elem<__nv_bfloat16>;
    const __nv_bfloat162 v =
        __hmax2_nan(__hmax2_nan(E::pair(w.x), E::pair(w.y)), __hmax2_nan(E::pair(w.z), E::pair(w.w)));
    m = first ? v : __hmax2_nan(m, v);
  }
  __device__ __forceinline__ void join(const VecMax& o, bool first) {
    m = first ? o.m : __hmax2_nan(m, o.m);
  }
  __device__ __forceinline__ float value() const {
    return fmax_nan(__low2float(m), __high2float(m));
  }
  __device__ __forceinline__ bool reaches(float tau) const {
    // (tau is a bfloat16 value; -inf: an entry above it)
    const float v = value();
    return v >= tau && v > -INFINITY;
  }
};

// The order-preserving key's value (f32_key's inverse).
__device__ __forceinline__ float f32_of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Index of this thread's vector u of tile i. A warp's vectors of one u are adjacent (512 bytes).
// Contiguous: a warp's kTileVecs pieces are adjacent, and so are the warps and the tiles.
// Interleaved: the pieces of the row are dealt out to the tiles in turn.
__device__ __forceinline__ int tile_vector_of(bool interleaved, int i, int n, int u, int warp,
                                              int lane) {
  return interleaved ? ((u * kWarps + warp) * n + i) * 32 + lane
                     : ((i * kWarps + warp) * kTileVecs + u) * 32 + lane;
}
__device__ __forceinline__ int tile_vector(bool interleaved, int i, int n, int u) {
  return tile_vector_of(interleaved, i, n, u, int(threadIdx.x >> 5), int(threadIdx.x & 31));
}

// Loads this thread's vectors of tile i of n (-inf past the row), all before any is used. Whole
// vectors are told by one unsigned comparison.
template <typename T, bool kOnce>
__device__ __forceinline__ void load_tile(const RowView<T, kOnce>& rv, bool interleaved, int i,
                                          int n, uint4 (&w)[kTileVecs]) {
  constexpr int P = Elem<T>::kPerVec;
  const int ga = rv.mis ? 1 : 0;                      // whole vectors: ga <= g < gb
  const unsigned span = unsigned((rv.V + rv.mis) / P - ga);
  const int g0 = tile_vector(interleaved, i, n, 0);
  const int step = interleaved ? n * kThreads : 32;
  const uint4* p = reinterpret_cast<const uint4*>(rv.row - rv.mis) + g0;
  if ((rv.V + rv.mis) / P < ga) {  // the row lies within one vector
#pragma unroll
    for (int u = 0; u < kTileVecs; ++u)
      w[u] = g0 + u * step < rv.G ? rv.load(g0 + u * step) : neg_inf_vec(int(sizeof(T)));
    return;
  }
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u)
    if (unsigned(g0 + u * step - ga) < span) w[u] = rv.get(p + u * step);
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    const int g = g0 + u * step;
    if (unsigned(g - ga) >= span) w[u] = g < rv.G ? rv.load(g) : neg_inf_vec(int(sizeof(T)));
  }
}

// The same into shared memory, asynchronously: this thread's vector u goes to
// sh[u kThreads + threadIdx.x], and only this thread reads it there, after tile_arrived().
template <typename T, bool kOnce>
__device__ __forceinline__ void fetch_tile(const RowView<T, kOnce>& rv, bool interleaved, int i,
                                           int n, uint4* sh) {
  constexpr int P = Elem<T>::kPerVec;
  const int ga = rv.mis ? 1 : 0, gb = max((rv.V + rv.mis) / P, ga);  // whole vectors: ga <= g < gb
  const int g0 = tile_vector(interleaved, i, n, 0);
  const int step = interleaved ? n * kThreads : 32;
  const uint4* p = reinterpret_cast<const uint4*>(rv.row - rv.mis) + g0;
  const uint32_t to = smem_u32(sh + threadIdx.x);
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u)
    if (unsigned(g0 + u * step - ga) < unsigned(gb - ga))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + u * kThreads * 16),
                   "l"(p + size_t(unsigned(u * step)))
                   : "memory");
  if (g0 < ga || g0 + (kTileVecs - 1) * step >= gb) {  // the row's ends: few threads, so kept small
#pragma unroll 1
    for (int u = 0; u < kTileVecs; ++u) {
      const int g = g0 + u * step;
      if (unsigned(g - ga) >= unsigned(gb - ga))
        sh[u * kThreads + threadIdx.x] = g < rv.G ? rv.load(g) : neg_inf_vec(int(sizeof(T)));
    }
  }
}
__device__ __forceinline__ void tile_arrived() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// This thread's vectors of a tile in shared memory.
struct TileRef {
  uint4* sh;
  __device__ __forceinline__ uint4& operator[](int u) const { return sh[u * kThreads]; }
};
// Entry e of a vector in memory.
template <typename T>
__device__ __forceinline__ float entry_of(const uint4& v, int e) {
  if constexpr (sizeof(T) == 4)
    return reinterpret_cast<const float*>(&v)[e];
  else
    return __uint_as_float(uint32_t(reinterpret_cast<const unsigned short*>(&v)[e]) << 16);
}

// Largest value over the warp; NaN if any lane holds NaN.
__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmax_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum_f32(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// log2(e) / T in two floats: hi just below it, lo the positive remainder. The remainder costs
// one packed multiply per two entries and takes away the error that is the same for all
// entries (a rounded c is another temperature); lo > 0 (a subnormal at least) keeps (-inf) * lo
// at -inf.
struct Log2Scale {
  float hi, lo;
};
// The largest scale that a float holds (a temperature below 2^-127 counts as about that).
constexpr double kMostScale = 3e38;
// On the host, for a call's one temperature.
inline Log2Scale log2_scale(double T) {
  const double c = fmin(1.4426950408889634074 / T, kMostScale);
  float hi = float(c);
  if (double(hi) >= c) hi = nextafterf(hi, 0.0f);
  return Log2Scale{hi, fmaxf(float(c - double(hi)), 1.4e-45f)};
}
// For a row's own temperature, in float32: hi is the rounded quotient less 2^-21 of it,
// lo the remainder, off by 2^-24 of itself (2^-46 of c).
__device__ __forceinline__ Log2Scale log2_scale_row(float T) {
  constexpr float L = 1.44269502f, Lr = 1.92596303e-8f;  // log2(e) = L + Lr
  if (!(T > 1.5e-30f && T < 1e30f)) {
    const double c = fmin(1.4426950408889634074 / double(T), kMostScale);
    const float h = __double2float_rd(c * (1.0 - 1e-7));
    return Log2Scale{h, fmaxf(float(c - double(h)), 1.4e-45f)};
  }
  const float q = __fdividef(L, T);
  const float hi = fmaf(q, -0x1p-21f, q);
  const float r = fmaf(-hi, T, L) + Lr;  // (the fma is exact to its one rounding)
  return Log2Scale{hi, __fdividef(r, T)};
}

// exp((x - m) / T) in float32, x <= m.
__device__ __forceinline__ float weight_f(float x, float m, const Log2Scale& c) {
  const float d = x - m;
  return ex2(fmaf(d, c.hi, d * c.lo));
}

// Sum of exp2((x - m) c) over the entries of one vector, m >= every entry and m > -inf. The
// difference is taken first: it is exact where it matters, and -inf or the type's lowest value
// minus m stays a number that weighs 0. Relative error of a weight: 2^-22 of ex2, and
// 2^-23 |x - m| c ln 2 of the two roundings of its argument.
template <typename T>
__device__ __forceinline__ float vec_exp_sum(const uint4& w, float m, const Log2Scale& c) {
  float x[Elem<T>::kPerVec];
  Elem<T>::unpack(w, x);
  const float2 nm = make_float2(-m, -m), hi = make_float2(c.hi, c.hi), lo = make_float2(c.lo, c.lo);
  const float2 zero = make_float2(0.0f, 0.0f);
  float2 s[Elem<T>::kPerVec / 2];
#pragma unroll
  for (int q = 0; q < Elem<T>::kPerVec / 2; ++q) {
    const float2 d = fadd2(make_float2(x[2 * q], x[2 * q + 1]), nm);
    const float2 y = ffma2(d, hi, ffma2(d, lo, zero));
    s[q] = make_float2(ex2(y.x), ex2(y.y));
  }
#pragma unroll
  for (int o = Elem<T>::kPerVec / 4; o > 0; o >>= 1)
#pragma unroll
    for (int q = 0; q < o; ++q) s[q] = fadd2(s[q], s[q + o]);
  return s[0].x + s[0].y;
}

// exp((x - m) / T) in double for x <= m, by the same table-driven method as exp_neg (Tang 1989)
// with the rounding to n done by adding 1.5 2^52, no branches and the table in shared memory:
// 3.1 entries per clock and SM against exp_neg's 1.8 (both bound by instruction issue; measured
// on 16 entries a thread). Weights below 2^-1000 are 0. Relative error a few units in the last
// place.
struct DoubleWeight {
  double md, c64;
  float m, least;     // x - m > least: weights above 2^-1000 (-inf where no float lies below that)
  const double* tab;  // 2^(j/64), 64 entries in shared memory
  __device__ __forceinline__ DoubleWeight(float m_, double iT, const double* tab_)
      : md(double(m_)), c64(iT * 92.33248261689366), m(m_),
        least(float(-1000.0 * 0.6931471805599453 / iT)), tab(tab_) {}
  __device__ __forceinline__ double operator()(float x) const {
    constexpr double kMagic = 6755399441055744.0;  // 1.5 2^52
    constexpr double L = 0.010830424696249145;     // ln2 / 64
    const double d = double(x) - md;
    const double y = fma(d, c64, kMagic);
    const int n = __double2loint(y);
    const double r = fma(d, c64, kMagic - y);
    double p = fma(r, L * L * L * L * L / 120.0, L * L * L * L / 24.0);
    p = fma(p, r, L * L * L / 6.0);
    p = fma(p, r, L * L / 2.0);
    p = fma(p, r, L);
    double t = tab[n & 63];
    t = fma(t, p * r, t);
    const bool on = x - m > least;
    return __hiloint2double(on ? __double2hiint(t) + ((n >> 6) << 20) : 0,
                            on ? __double2loint(t) : 0);
  }
};
__device__ __forceinline__ void load_exp_table(double* tab) {
  if (threadIdx.x < 64) tab[threadIdx.x] = kExp2J[threadIdx.x];
}

}  // namespace sv

// Distillation from a teacher's top logits: the loss of a student's logit rows and its gradient.
//
// Row r lists up to k of the teacher's entries (ids i_j, logits a_j; entries with a negative id
// or a logit of -inf are padding). With temperature T, the student's s = softmax(z / T), and
//   t_j = softmax over the list of a_j / T, rho = 0            (no teacher lse), or
//   t_j = exp(a_j / T - lse), rho = 1 - sum_j t_j              (the teacher's own log-sum-exp),
// rho being the teacher's mass outside the list (0 where it lies within the rounding of a float32
// lse, (|lse| + 1) 2^-23) and sigma the student's:
//   L = sum_j t_j (log t_j - log s_{i_j}) + rho (log rho - log sigma)
//   dL/dz_v = (s_v - t_v) / T listed,  (sigma - rho) q_v / T unlisted,
// q_v = s_v / sigma the student's share of its own rest. That is L's derivative where
// M = sum_j t_j + rho is 1; where an lse too small for its list makes M larger (rho is held at 0), the
// loss counts its sum t_j and the gradient still counts 1. sigma comes from the sum over the
// unlisted entries alone, never from 1 - sum_j s_{i_j}, which cancels when the student is sure.
//
// What bounds it: HBM. The loss reads a row once, the gradient reads and writes it once; the
// exponentials ask for 0.7 of the SFU's rate at the HBM rate of bfloat16 rows. Measured, bfloat16:
// sums of 2,048 x 32,000 27 us (4.8 TB/s), gradient of 1,024 x 151,936 103 us (6.0 TB/s), both at
// once of 2,048 x 128,256 240 us (4.4 TB/s read and written; by the two calls 96 + 13 + 158).
#pragma once

#include <type_traits>

#include "rowtile.cuh"

namespace sv {

constexpr int kMaxTeacher = 256;     // entries of a teacher's list

// What one warp of a tile saw of the unlisted entries: the largest (NaN: an entry is NaN or +inf,
// or the row's list is in error) and the sum of exp((z - m) / T).
struct DistillPart {
  float m, s;
};

struct DistillJob {
  const void* logits;
  long long stride;
  int rows, V, n, k;
  double iT;
  Log2Scale c;
  const int32_t* ids;       // [rows][k]
  const float* values;      // [rows][k]
  const float* lse;         // [rows] or NULL
  DistillPart* parts;       // [rows][n][kWarps]
  float* loss;              // [rows]
  float* stats;             // [rows][4]
};

struct DistillGradJob {
  const void* logits;
  long long stride;
  int rows, V, n, k;
  float temp;
  Log2Scale c;
  const int32_t* ids;
  const float* values;
  const float* lse;
  const float* stats;       // [rows][4]
  const float* grad_loss;   // [rows] or NULL (1)
  void* grad;
  long long grad_stride;
};

__device__ __forceinline__ bool teacher_used(int id, float v) { return id >= 0 && !(v == -INFINITY); }

// Marks the listed entries of a contiguous tile in a byte per vector; id is the thread's list entry
// (-1: none). Returns whether an id of the row is out of range, or (seen where it stands) twice
// there. Two barriers.
template <typename T, bool kOnce>
__device__ __forceinline__ int mark_listed(uint32_t* marks, const RowView<T, kOnce>& rv, int tile,
                                           int id) {
  constexpr int P = Elem<T>::kPerVec;
  for (int i = threadIdx.x; i < kTileVectors / 4; i += kThreads) marks[i] = 0u;
  __syncthreads();
  int bad = 0;
  if (id >= 0) {
    const unsigned at = unsigned(id + rv.mis) - unsigned(tile) * unsigned(kTileVectors * P);
    if (id >= rv.V) {
      bad = 1;
    } else if (at < unsigned(kTileVectors * P)) {
      const uint32_t v = at / P, bit = 1u << ((v & 3u) * 8u + at % P);
      if (atomicOr(&marks[v >> 2], bit) & bit) bad = 1;
    }
  }
  return __syncthreads_or(bad);
}

// The warp's part of a tile: its marked entries become -inf in w (the loss looks at them by
// themselves), the others give the maximum and the weight sum. w[u] is this thread's vector u, in
// registers or (TileRef) in shared memory.
template <typename T, typename Tile>
__device__ __forceinline__ DistillPart weigh_unlisted(const uint32_t* marks, Tile&& w,
                                                      const Log2Scale& c, int bad) {
  constexpr int P = Elem<T>::kPerVec;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint8_t* mine = reinterpret_cast<const uint8_t*>(marks) + warp * kTileVecs * 32 + lane;
  VecMax<T> mx;
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    const uint32_t b = mine[u * 32];
    uint4 x = w[u];
    if (b) {
      uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (b >> e & 1u) {
          if constexpr (sizeof(T) == 4)
            v[e] = 0xFF800000u;
          else
            v[e >> 1] = (e & 1) ? (v[e >> 1] & 0xFFFFu) | 0xFF800000u
                                : (v[e >> 1] & 0xFFFF0000u) | 0xFF80u;
        }
      w[u] = x = make_uint4(v[0], v[1], v[2], v[3]);
    }
    mx.add(x, u == 0);
  }
  const float m = warp_max_nan(mx.value());
  float s = 0.0f;
  if (m > -INFINITY && m < INFINITY) {
    float f[kTileVecs];
#pragma unroll
    for (int u = 0; u < kTileVecs; ++u) f[u] = vec_exp_sum<T>(w[u], m, c);
#pragma unroll
    for (int o = kTileVecs / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < o; ++u) f[u] += f[u + o];
    s = warp_sum_f32(f[0]);
  }
  return DistillPart{(bad || !(m < INFINITY)) ? NAN : m, s};
}

// One contiguous tile of a row: each warp's maximum and weight sum of the unlisted entries. The
// marks are made while the tile's loads are under way (into shared memory: six blocks an SM; with the
// tile in registers four fit, and 2,048 x 32,000 took 2 us longer than its 27); from there on each
// warp works and answers by itself.
template <typename T>
__global__ void __launch_bounds__(kThreads, 6) distill_tile_kernel(const DistillJob j) {
  __shared__ __align__(16) uint4 s_tile[kTileVectors];
  __shared__ uint32_t s_marks[kTileVectors / 4];
  const int n = j.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = int(blockIdx.x / unsigned(n)), tile = int(blockIdx.x % unsigned(n));
  const RowView<T> rv(j.logits, row, j.stride, j.V);
  fetch_tile(rv, false, tile, n, s_tile);
  const TileRef w = {s_tile + tid};
  int id = -1;
  if (tid < j.k) {
    id = j.ids[size_t(row) * j.k + tid];
    if (!teacher_used(id, j.values[size_t(row) * j.k + tid])) id = -1;
  }
  const int bad = mark_listed(s_marks, rv, tile, id);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tile_arrived();
  const DistillPart p = weigh_unlisted<T>(s_marks, w, j.c, bad);
  if (lane == 0) j.parts[(size_t(row) * n + tile) * kWarps + warp] = p;
}

__device__ __forceinline__ float warp_max_f32(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// The student's side of a row that the loss and the gradient share.
struct StudentRow {
  float m, m_rest;  // largest logit; largest unlisted one
  double Z, R;      // sums of exp((z - m) / T) over all entries, exp((z - m_rest) / T) over the rest
};

// What the list alone gives of a row.
struct ListSide {
  double log_t;   // t_j = exp(a_j / T - log_t)
  double mass;    // sum of t_j
  double rho;     // the teacher's mass outside the list
  double cross;   // sum of t_j (log t_j - x_j / T), x_j the student's logits
  float xm;       // the largest x_j (-inf: none)
  float zs;       // sum of exp((x_j - xm) / T)
  int32_t flags;  // 1: the row is in error, 2: the list has an entry
  int32_t pad;
};
static_assert(sizeof(ListSide) == 48, "ListSide is 48 bytes");

// The list of a row by one warp. z(id) gives the student's logit of an entry.
template <typename Z>
__device__ __forceinline__ ListSide weigh_list(int k, double iT, const int32_t* ids,
                                               const float* values, const float* lse, Z&& z) {
  constexpr int kPer = kMaxTeacher / 32;
  const int lane = threadIdx.x & 31;
  int id[kPer];
  float a[kPer], x[kPer];
  // all ids, then all logits, under way together
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = q * 32 + lane;
    id[q] = i < k ? ids[i] : -1;
    a[q] = i < k ? values[i] : -INFINITY;
  }
  float am = -INFINITY, xm = -INFINITY;
  int bad = 0, any = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    x[q] = -INFINITY;
    if (!teacher_used(id[q], a[q])) {
      id[q] = -1;
      a[q] = -INFINITY;
    } else {
      x[q] = z(id[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (id[q] >= 0) {
      any = 1;
      bad |= !(a[q] < INFINITY) || !(x[q] < INFINITY);
      am = fmaxf(am, a[q]);
      xm = fmaxf(xm, x[q]);
    }
  am = warp_max_f32(am);
  xm = warp_max_f32(xm);
  bad = __any_sync(0xffffffffu, bad);
  any = __any_sync(0xffffffffu, any);
  ListSide l = {0.0, 0.0, 0.0, 0.0, xm, 0.0f, any ? 2 : 0, 0};
  double ta = 0.0, zs = 0.0, ex = 0.0;
  if (!bad && any) {
    // weights relative to the largest; entries past the list have weight 0
#pragma unroll 1
    for (int q = 0; q * 32 < k; ++q) {
      float aq = a[0], xq = x[0];
#pragma unroll
      for (int u = 1; u < kPer; ++u)
        if (u == q) {
          aq = a[u];
          xq = x[u];
        }
      const double t = weight_d(aq, am, iT);
      ta += t;
      if (xq > -INFINITY) zs += weight_d(xq, xm, iT);
      if (t > 0.0) ex += t * ((double(aq) - double(xq)) * iT);
    }
    ta = warp_sum_f64(ta);
    zs = warp_sum_f64(zs);
    ex = warp_sum_f64(ex);
  }
  l.zs = float(zs);
  double scale = 0.0;  // t_j = weight_j scale
  if (lse) {
    l.log_t = double(*lse);
    if (!(fabs(l.log_t) < INFINITY)) bad = 1;
    scale = any ? exp(double(am) * iT - l.log_t) : 0.0;
    l.mass = ta * scale;
    l.rho = 1.0 - l.mass;
    // (a list without entries asks for nothing: no rest either)
    if (!any || !(l.rho > (fabs(l.log_t) + 1.0) * 0x1.0p-23)) l.rho = 0.0;
  } else if (any) {
    l.log_t = double(am) * iT + log(ta);
    scale = 1.0 / ta;
    l.mass = 1.0;
  }
  // sum t (a / T - x / T) - log_t sum t (scale 0: all masses are below a double's smallest, and a
  // masked x asks for nothing)
  l.cross = any && scale > 0.0 ? ex * scale - l.log_t * l.mass : 0.0;
  l.flags |= bad ? 1 : 0;
  return l;
}

// A row's loss and statistics in double, by one warp, from its n parts and its list's side.
__device__ __forceinline__ void finish_loss(const DistillPart* parts, int n, double iT,
                                            const ListSide* l, bool tail, float* loss,
                                            float* stats) {
  const int lane = threadIdx.x & 31;
  float mr = -INFINITY;
  int bad = l->flags & 1;
#pragma unroll 1
  for (int i = lane; i < n; i += 32) {
    const float p = parts[i].m;
    bad |= !(p == p);
    mr = fmaxf(mr, p);
  }
  mr = warp_max_f32(mr);
  const float xm = l->xm, m = fmaxf(mr, xm);
  const bool any = (l->flags & 2) != 0;
  const bool inv = __any_sync(0xffffffffu, bad) || !(m > -INFINITY);
  double R = 0.0, part = 0.0, Z = 0.0;
  if (!inv) {
#pragma unroll 1
    for (int i = lane; i < n; i += 32) {
      const DistillPart p = parts[i];
      if (p.m > -INFINITY) R += double(p.s) * weight_d(p.m, mr, iT);
    }
    R = warp_sum_f64(R);
    Z = (any && xm > -INFINITY ? double(l->zs) * weight_d(xm, m, iT) : 0.0) +
        (mr > -INFINITY ? R * weight_d(mr, m, iT) : 0.0);
    const double log_z = double(m) * iT + log(Z);
    part = any ? l->cross + l->mass * log_z : 0.0;
    if (tail && l->rho > 0.0) {
      const double log_sigma = R > 0.0 ? double(mr) * iT + log(R) - log_z : -INFINITY;
      part += l->rho * (log(l->rho) - log_sigma);
    }
  }
  if (lane == 0) {
    *loss = inv ? NAN : float(part);
    if (stats)
      *reinterpret_cast<float4*>(stats) = inv ? make_float4(NAN, NAN, NAN, NAN)
                                              : make_float4(m, float(Z), mr, float(R));
  }
}

// One warp per row, after distill_tile_kernel. Its blocks start as the last tiles end (the tiles'
// kernel lets them) and weigh the lists meanwhile.
template <typename T>
__global__ void __launch_bounds__(kThreads) distill_finish_kernel(
    const __grid_constant__ DistillJob j) {
  __shared__ ListSide s_list[kWarps];
  const int warp = threadIdx.x >> 5, row = int(blockIdx.x) * kWarps + warp;
  if (row < j.rows) {
    const RowView<T> rv(j.logits, row, j.stride, j.V);
    const ListSide l = weigh_list(j.k, j.iT, j.ids + size_t(row) * j.k,
                                  j.values + size_t(row) * j.k, j.lse ? j.lse + row : nullptr,
                                  [&](int i) { return i < j.V ? rv.entry(i) : 0.0f; });
    if ((threadIdx.x & 31) == 0) s_list[warp] = l;
    __syncwarp();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row < j.rows)
    finish_loss(j.parts + size_t(row) * j.n * kWarps, j.n * kWarps, j.iT, &s_list[warp],
                j.lse != nullptr, j.loss + row, j.stats ? j.stats + size_t(row) * 4 : nullptr);
}

// Gradient entries of one vector of unlisted logits: exp2((z - m_rest) c) f.
template <typename T>
__device__ __forceinline__ void grad_vec(const uint4& w, float mr, const Log2Scale& c, float f,
                                         float* o) {
  float x[Elem<T>::kPerVec];
  Elem<T>::unpack(w, x);
  const float2 nm = make_float2(-mr, -mr), hi = make_float2(c.hi, c.hi), lo = make_float2(c.lo, c.lo);
  const float2 zero = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int q = 0; q < Elem<T>::kPerVec / 2; ++q) {
    const float2 d = fadd2(make_float2(x[2 * q], x[2 * q + 1]), nm);
    const float2 y = ffma2(d, hi, ffma2(d, lo, zero));
    o[2 * q] = ex2(y.x) * f;
    o[2 * q + 1] = ex2(y.y) * f;
  }
}

template <typename T>
__device__ __forceinline__ void store_one(T* p, float x) {
  if constexpr (sizeof(T) == 4)
    *p = x;
  else
    *p = __float2bfloat16_rn(x);
}

template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float* o) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                      __float_as_uint(o[3]));
  } else {
    uint32_t v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * q], o[2 * q + 1]);
      v[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// Writes the gradient entries of this thread's vectors of a contiguous tile as unlisted ones (0 when
// zero is set). The output row may stand differently on the 16-byte grid: then entries are stored
// one by one.
template <typename T, bool kOnce, typename Tile>
__device__ __forceinline__ void store_unlisted(const RowView<T, kOnce>& rv, T* out, int tile, int n,
                                               const Tile& w, float mr, const Log2Scale& c, float f,
                                               bool zero) {
  constexpr int P = Elem<T>::kPerVec;
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15u) ==
                    (reinterpret_cast<uintptr_t>(rv.row) & 15u);
  const int v0 = tile_vector(false, tile, n, 0);
  const int ga = rv.mis ? 1 : 0, gb = (rv.V + rv.mis) / P;  // whole vectors: ga <= v < gb
  if (same && v0 >= ga && v0 + (kTileVecs - 1) * 32 < gb) {
    // all of this thread's vectors are whole: eight aligned stores
    uint4* to = reinterpret_cast<uint4*>(out - rv.mis) + v0;
    if (zero) {
#pragma unroll
      for (int u = 0; u < kTileVecs; ++u) to[u * 32] = make_uint4(0u, 0u, 0u, 0u);
      return;
    }
#pragma unroll
    for (int u = 0; u < kTileVecs; ++u) {
      float o[P];
      grad_vec<T>(w[u], mr, c, f, o);
      to[u * 32] = pack_vec<T>(o);
    }
    return;
  }
  auto one = [&](int u) {
    const int v = v0 + u * 32;
    if (v >= rv.G) return;
    float o[P];
#pragma unroll
    for (int e = 0; e < P; ++e) o[e] = 0.0f;
    if (!zero) grad_vec<T>(w[u], mr, c, f, o);
    const int e0 = rv.first(v);
    if (same && rv.whole(v)) {
      *reinterpret_cast<uint4*>(out + e0) = pack_vec<T>(o);
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (e0 + e >= 0 && e0 + e < rv.V) store_one(out + e0 + e, o[e]);
    }
  };
  if constexpr (std::is_same<Tile, TileRef>::value) {
#pragma unroll 1
    for (int u = 0; u < kTileVecs; ++u) one(u);  // (unrolled, its code slows the row kernel by 8 %)
  } else {
#pragma unroll
    for (int u = 0; u < kTileVecs; ++u) one(u);
  }
}

// The factors of a row's gradient: f of the unlisted entries (times exp((z - m_rest) / T)), and
// g / T, 1 / Z for the listed ones. A list with no entries asks for nothing: f = 0.
struct GradRow {
  float f, m_rest;
  double gT, iZ;
};

__device__ __forceinline__ GradRow grad_row(const StudentRow& st, double rho, bool any, double g,
                                            float temp) {
  GradRow r;
  const double iT = 1.0 / double(temp);
  r.gT = g * iT;
  r.iZ = 1.0 / st.Z;
  const bool none = st.R == 0.0;  // no unlisted entry has mass: their gradients are 0
  const double sigma = none ? 0.0 : st.R * weight_d(st.m_rest, st.m, iT) * r.iZ;
  r.f = (none || !any) ? 0.0f : float(r.gT * (sigma - rho) / st.R);
  if (!(st.Z == st.Z)) r.f = NAN;  // a row in error
  r.m_rest = none ? 0.0f : st.m_rest;
  return r;
}

// One contiguous tile of a row. The tile's entries are written as unlisted ones; then each
// listed entry of the tile is written by the thread that holds it in the list, which read its
// logit before the first store (grad may be logits). Every block of a row weighs the list again,
// under its own loads: 103 us for 1,024 x 151,936, 0.92 of a plain copy.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) distill_grad_kernel(const DistillGradJob j) {
  constexpr int P = Elem<T>::kPerVec;
  __shared__ double s_scr[kWarps];
  __shared__ float s_scr_f[kWarps];
  const int n = j.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = int(blockIdx.x / unsigned(n)), tile = int(blockIdx.x % unsigned(n));
  const RowView<T, false> rv(j.logits, row, j.stride, j.V);
  T* out = static_cast<T*>(j.grad) + (long long)row * j.grad_stride;
  const float g = j.grad_loss ? j.grad_loss[row] : 1.0f;
  uint4 w[kTileVecs];
  if (g != 0.0f) load_tile(rv, false, tile, n, w);
  // the list: every block of the row weighs it, while its loads are under way
  const double iT = 1.0 / double(j.temp);
  int id = -1;
  float a = -INFINITY, x = 0.0f;
  if (tid < j.k) {
    id = j.ids[size_t(row) * j.k + tid];
    a = j.values[size_t(row) * j.k + tid];
    if (!teacher_used(id, a)) id = -1;
  }
  const bool here = id >= 0 && id < j.V &&
                    (id + rv.mis) / (kTileVectors * P) == tile;
  GradRow gr = {0.0f, 0.0f, 0.0, 0.0};
  double t = 0.0;
  const float4 s4 = reinterpret_cast<const float4*>(j.stats)[row];
  const StudentRow st = {s4.x, s4.z, double(s4.y), double(s4.w)};
  if (g != 0.0f) {
    if (here) x = rv.entry(id);
    const int any = __syncthreads_or(id >= 0);
    double rho = 0.0;
    if (j.lse) {
      const double l = double(j.lse[row]);
      t = id >= 0 ? exp(double(a) * iT - l) : 0.0;
      rho = 1.0 - block_sum_f64(t, s_scr);
      if (!(rho > (fabs(l) + 1.0) * 0x1.0p-23)) rho = 0.0;
    } else {
      float am = warp_max_f32(id >= 0 ? a : -INFINITY);
      if (lane == 0) s_scr_f[warp] = am;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kWarps; ++q) am = fmaxf(am, s_scr_f[q]);
      t = id >= 0 ? weight_d(a, am, iT) : 0.0;
      const double all = block_sum_f64(t, s_scr);
      t = id >= 0 ? t / all : 0.0;
    }
    gr = grad_row(st, rho, any != 0, double(g), j.temp);
  }
  store_unlisted(rv, out, tile, n, w, gr.m_rest, j.c, gr.f, g == 0.0f);
  if (g == 0.0f) return;  // (uniform)
  __syncthreads();
  if (here) store_one(out + id, float(gr.gT * (weight_d(x, st.m, iT) * gr.iZ - t)));
}

// ------------------------------------------------------------------------- whole rows at once
// Rows of up to sixteen tiles: a cluster holds a row in shared memory, a tile per block, so that
// the row is read once for both its sum and its gradient, and the loss takes one launch. The blocks
// exchange their warps' maxima and sums through distributed shared memory and each works out the
// row's factors; the list's side of them is done while the tile's loads are under way. The blocks
// wait at the cluster's barrier for about half their time (issue slots 60% busy).
constexpr int kMaxRowBlocks = 16;

struct DistillRowJob {
  const void* logits;
  long long stride;
  int rows, V, n, k;
  double iT;
  Log2Scale c;
  const int32_t* ids;
  const float* values;
  const float* lse;
  const float* grad_loss;
  float* loss;
  float* stats;         // [rows][4] or NULL
  void* grad;
  long long grad_stride;
  struct ListSide* lists;  // [rows]
};

template <typename T>
__global__ void __launch_bounds__(kThreads) distill_list_kernel(
    const __grid_constant__ DistillRowJob j) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = int(blockIdx.x) * kWarps + int(threadIdx.x >> 5);
  if (row >= j.rows) return;
  const RowView<T> rv(j.logits, row, j.stride, j.V);
  const ListSide l = weigh_list(j.k, j.iT, j.ids + size_t(row) * j.k,
                                j.values + size_t(row) * j.k, j.lse ? j.lse + row : nullptr,
                                [&](int i) { return i < j.V ? rv.entry(i) : 0.0f; });
  if ((threadIdx.x & 31) == 0) j.lists[row] = l;
}

// A block may write to another's shared memory only once that one runs: each says so as it starts, and
// waits for its fellows before its first remote store, behind its list and under its tile's loads.
// (Nothing is handed over here, so that the arrival is relaxed; the exchange has a barrier of its own.)
__device__ __forceinline__ void cluster_arrive_started() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_started() {
  asm volatile("barrier.cluster.wait;" ::: "memory");
}

struct DistillRowSmem {
  uint32_t marks[kTileVectors / 4];
  DistillPart part[kMaxRowBlocks * kWarps];  // the row's, in every block
  ListSide list;
};

// A block does its tile's sums and sends its warps' parts to every block of the cluster; after the
// exchange's barrier every warp puts the row together for itself from its own block's shared
// memory, in float32: the gradient's factors need no more, nor does the loss beside them. The
// list's side comes from distill_list_kernel, which runs beside the tiles' loads (kList false),
// or, in calls too small for a second launch to pay, from the first block's first warp (it would
// hold up the cluster: 4 us of a block's 10).
template <typename T, bool kGrad, bool kList>
__global__ void __launch_bounds__(kThreads, 6) distill_row_kernel(
    const __grid_constant__ DistillRowJob j) {
  __shared__ DistillRowSmem sm;
  __shared__ __align__(16) uint4 s_tile[kTileVectors];
  cluster_arrive_started();
  cg::cluster_group cl = cg::this_cluster();
  const int n = j.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = int(blockIdx.x / unsigned(n)), tile = int(blockIdx.x % unsigned(n));
  const RowView<T, !kGrad> rv(j.logits, row, j.stride, j.V);
  fetch_tile(rv, false, tile, n, s_tile);
  const TileRef w = {s_tile + tid};
  int id = -1;
  float a = -INFINITY;
  if (tid < j.k) {
    id = j.ids[size_t(row) * j.k + tid];
    a = j.values[size_t(row) * j.k + tid];
    if (!teacher_used(id, a)) id = -1;
  }
  const bool here = id >= 0 && id < j.V &&
                    (id + rv.mis) / (kTileVectors * Elem<T>::kPerVec) == tile;
  float x = 0.0f;
  if (kGrad && here) x = rv.entry(id);
  const int bad = mark_listed(sm.marks, rv, tile, id);
  const int to = kGrad ? n : 1;  // blocks that need the row's parts
  cluster_wait_started();
  if (kList && tile == 0 && warp == 0) {
    const ListSide l = weigh_list(j.k, j.iT, j.ids + size_t(row) * j.k,
                                  j.values + size_t(row) * j.k, j.lse ? j.lse + row : nullptr,
                                  [&](int i) { return i < j.V ? rv.entry(i) : 0.0f; });
    if (lane < to) cl.map_shared_rank(&sm, unsigned(lane))->list = l;
  }
  tile_arrived();
  const DistillPart mine = weigh_unlisted<T>(sm.marks, w, j.c, bad);
  if (lane < to) cl.map_shared_rank(&sm, unsigned(lane))->part[tile * kWarps + warp] = mine;
  const float g = kGrad && j.grad_loss ? j.grad_loss[row] : 1.0f;
  const float gT = g * float(j.iT);  // (g 0: not looked at, 1 / T may be infinite here)
  if (!kList) asm volatile("griddepcontrol.wait;" ::: "memory");
  const ListSide* l = kList ? &sm.list : j.lists + row;
  ListSide ls;
  if (kGrad && !kList) ls = *l;  // (before the barrier: its latency is the cluster's)
  cl.sync();
  if (!kGrad && (tile != 0 || warp != 0)) return;
  float mr = -INFINITY, m = 0.0f, iZ = 0.0f, R = 0.0f;
  if constexpr (kGrad) {
    if (kList) ls = *l;
    // the row's factors
    const bool any = (ls.flags & 2) != 0;
    constexpr int kPer = kMaxRowBlocks * kWarps / 32;
    DistillPart p[kPer];
    bool inv = (ls.flags & 1) != 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = q * 32 + lane;
      p[q] = i < n * kWarps ? sm.part[i] : DistillPart{-INFINITY, 0.0f};
      inv |= !(p[q].m == p[q].m);
      mr = fmaxf(mr, p[q].m);
    }
    mr = warp_max_f32(mr);
    m = fmaxf(mr, ls.xm);
    inv = __any_sync(0xffffffffu, inv) || !(m > -INFINITY);
    const bool none = !(mr > -INFINITY);
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (p[q].m > -INFINITY) R += p[q].s * weight_f(p[q].m, mr, j.c);
    R = warp_sum_f32(R);
    const float rest = none ? 0.0f : R * weight_f(mr, m, j.c);
    iZ = 1.0f / (rest + (any && ls.xm > -INFINITY ? ls.zs * weight_f(ls.xm, m, j.c) : 0.0f));
    const float f = inv ? NAN : ((none || !any) ? 0.0f : gT * (rest * iZ - float(ls.rho)) / R);
    if (inv) iZ = NAN;
    if (none) mr = 0.0f;
    T* out = static_cast<T*>(j.grad) + (long long)row * j.grad_stride;
    store_unlisted(rv, out, tile, n, w, mr, j.c, f, g == 0.0f);
    __syncthreads();
    if (here && g != 0.0f) {
      // (the exponent in double: a_j / T and log_t may be large and near each other)
      const float t = ex2(float((double(a) * j.iT - ls.log_t) * 1.4426950408889634));
      const float s = (x > -INFINITY ? weight_f(x, m, j.c) : 0.0f) * iZ;  // NaN: in error
      store_one(out + id, gT * (s - t));
    }
  }
  if constexpr (!kGrad) {
    finish_loss(sm.part, n * kWarps, j.iT, l, j.lse != nullptr, j.loss + row,
                j.stats ? j.stats + size_t(row) * 4 : nullptr);
  } else if (tile == 0 && tid == 0) {
    // The loss from the same float32 sums. R and Z are off by up to 2.6e-6 of themselves from the
    // tiles (2^-22 + 11 2^-24 + 8.3e-8 log2(V / sum)) and 1.2e-6 from putting up to 128 parts
    // together, an absolute error of their logarithms: under 4e-6 (mass + 2 rho) of the loss.
    const double log_z = double(m) * j.iT - log(double(iZ));
    double loss = (l->flags & 2) ? l->cross + l->mass * log_z : 0.0 * log_z;
    if (j.lse && l->rho > 0.0) {
      const double log_sigma = R > 0.0f ? double(mr) * j.iT + log(double(R)) - log_z : -INFINITY;
      loss += l->rho * (log(l->rho) - log_sigma);
    }
    j.loss[row] = float(loss);
  }
}

}  // namespace sv

// expert_dense.inl -- the experts' fully connected layers over rows sorted by expert, on the
// matrix cores.  Part of the translation unit of dense.hip.
//
// Expert e has the sorted positions p in [offsets[e], offsets[e+1]) and the weights W[e]
// [N, K].  With x(p) = X[p], or the token's row X[order[p] / k] read in place:
//   forward   Y[p, :]  = act(W[e] x(p) + b[e])
//   backward  dX[p, :] = W[e]^T dY[p, :], times [x(p) > 0] where x is a rectified output
//             dW[e]    = sum_p dY[p, :] x(p)^T,   db[e] = sum_p dY[p, :]        (fp32)
// Three products of one shape: rows by columns over a reduction, the rows cut at the experts'
// borders.  The row counts stay on the device: the grid has a block for every tile that n
// rows in E pieces can need, and a block finds its expert by a scan over the offsets.
// Positions from offsets[E] on belong to no expert; their rows of Y and dX are zero.
// Products are exact in the matrix cores (binary32 operands: rounded once), sums are fp32.
#include <cstdlib>
namespace ctr {
namespace experts {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

struct Product {
  const void* X;
  int64_t xs, x_rows;
  const int32_t* order;         // nullable: positions are X's rows
  uint32_t kmul;                // i / k = 2 i * kmul >> 32 + kshift for 0 <= i < 2^31
  int kshift;
  const int32_t* offsets;
  int64_t n;
  int E, K, N;
  const void* W;
  const float* b;               // forward, nullable
  int relu;                     // forward: act; backward: x is a rectified output
  const void* dY;
  int64_t dys;
  void* Y;                      // Y, or dX
  int64_t ys;
  float* dW;
  float* part;                  // partial sums of dW
  int64_t slice;                // positions a slice of dW's reduction
  bool slice_big;               //   in 256 x 256 tiles
  int col_tiles, row_tiles;
};

// First and last position of expert e; e == E: the positions of no expert.  Clamped, so that
// bad offsets give bad numbers and no access outside the arrays.
__device__ __forceinline__ void bounds_of(const Product& g, int e, int64_t* lo, int64_t* hi) {
  const int64_t a = clamp64(g.offsets[e], 0, g.n);
  *lo = a;
  *hi = e < g.E ? clamp64(g.offsets[e + 1], a, g.n) : g.n;
}

// The expert of row tile `mt` (BM rows a tile, experts in order, then the positions of none)
// and its rows: every wave scans the tile counts, 64 experts at a time.  false: no such tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const Product& g, int64_t mt, int* expert, int64_t* row0,
                                          int64_t* end) {
  const int lane = threadIdx.x & 63;
  int64_t run = 0;
  for (int e0 = 0; e0 <= g.E; e0 += 64) {
    const int e = e0 + lane;
    int64_t lo = 0, hi = 0;
    if (e <= g.E) bounds_of(g, e, &lo, &hi);
    const int tiles = (int)((hi - lo + BM - 1) / BM);
    int upto = tiles;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    const uint64_t past = __ballot(run + upto > mt);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      const int64_t first = run + __shfl(upto - tiles, at);
      *expert = e0 + at;
      *row0 = __shfl(lo, at) + (mt - first) * BM;
      *end = __shfl(hi, at);
      return true;
    }
    run += __shfl(upto, 63);
  }
  return false;
}

// Row of X of slot i (its token, i / k), or -1 (a slot outside X: its row reads as zeros).
__device__ __forceinline__ int32_t token_of(const Product& g, int32_t i) {
  const int32_t r = (int32_t)(__umulhi(2u * (uint32_t)i, g.kmul) >> g.kshift);
  return i >= 0 && r < (int32_t)g.x_rows ? r : -1;
}
// Row of X that position p reads, or -1.
__device__ __forceinline__ int64_t x_row(const Product& g, int64_t p) {
  if (!g.order) return p < g.x_rows ? p : -1;
  return token_of(g, g.order[p]);
}

template <int TY>
using Lds = typename std::conditional<TY == kEltF32, float, uint16_t>::type;

// Eight elements of one operand row, as stored, from base[off ..]; those at or past `left`
// are zero.
template <int TY>
struct Eight {
  Lds<TY> v[8];
  __device__ __forceinline__ void load(const void* base, int64_t off, int64_t left, bool vec) {
    const Lds<TY>* p = static_cast<const Lds<TY>*>(base) + off;
    if (vec && left >= 8) {
      if constexpr (TY == kEltF32) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        v[0] = (uint16_t)a.x; v[1] = (uint16_t)(a.x >> 16);
        v[2] = (uint16_t)a.y; v[3] = (uint16_t)(a.y >> 16);
        v[4] = (uint16_t)a.z; v[5] = (uint16_t)(a.z >> 16);
        v[6] = (uint16_t)a.w; v[7] = (uint16_t)(a.w >> 16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < left ? p[e] : Lds<TY>(0);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = Lds<TY>(0);
  }
};

enum Kind { kForward = 0, kInput = 1, kWeight = 2 };

// The product for any type, width, stride and alignment: a block has a 64 x 64 tile, each of
// its four waves a 32 x 32 matrix-core tile; the reduction advances 32 at a time through LDS.
template <int TY, int KIND>
__global__ __launch_bounds__(kThreads) void product_kernel(Product g) {
  using LT = Lds<TY>;
  constexpr int BM = 64, KT = 32, PITCH = TY == kEltF32 ? KT + 4 : KT + 8;
  __shared__ __attribute__((aligned(16))) LT As[BM * PITCH], Bs[BM * PITCH];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int wm = w >> 1, wn = w & 1, rl = lane & 31, kg = lane >> 5;
  const int n0 = (int)(blockIdx.x % g.col_tiles) * 64;
  const int64_t mt = blockIdx.x / g.col_tiles;
  const int cols = KIND == kForward ? g.N : g.K;
  int e;
  int64_t row0, end, r0 = 0, r1 = 0;       // output rows; reduction range
  if constexpr (KIND == kWeight) {
    e = (int)(mt / g.row_tiles);
    row0 = (mt % g.row_tiles) * BM;
    end = g.N;
    bounds_of(g, e, &r0, &r1);
  } else {
    if (!find_tile<BM>(g, mt, &e, &row0, &end)) return;
    r1 = e < g.E ? (KIND == kForward ? g.K : g.N) : 0;
  }
  const int elem = TY == kEltF32 ? 4 : 2;
  const int64_t we = (int64_t)e * g.N * g.K;           // e == E: not read
  const char* W = static_cast<const char*>(g.W) + we * elem;
  auto vec_ok = [&](const void* p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride * elem % 16 == 0;
  };
  const bool xv = vec_ok(g.X, g.xs), wv = vec_ok(W, g.K), yv = vec_ok(g.dY, g.dys);

  f32x16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.f;

  for (int64_t k0 = r0; k0 < r1; k0 += KT) {
    Eight<TY> a, b;
    // operands whose rows run along the reduction: row t / 4, elements 8 (t % 4) ..
    const int kr = t >> 2, kk = 8 * (t & 3);
    // operands whose rows are the reduction: row t / 8, elements 8 (t % 8) ..
    const int rr = t >> 3, rc = 8 * (t & 7);
    if constexpr (KIND == kForward) {
      const int64_t x = row0 + kr < end ? x_row(g, row0 + kr) : -1;
      if (x >= 0) a.load(g.X, x * g.xs + k0 + kk, r1 - k0 - kk, xv);
      else a.zero();
    } else if constexpr (KIND == kInput) {
      if (row0 + kr < end) a.load(g.dY, (row0 + kr) * g.dys + k0 + kk, r1 - k0 - kk, yv);
      else a.zero();
    } else {
      if (k0 + rr < r1) a.load(g.dY, (k0 + rr) * g.dys + row0 + rc, end - row0 - rc, yv);
      else a.zero();
    }
    if constexpr (KIND == kForward) {
      if (n0 + kr < cols) b.load(W, (int64_t)(n0 + kr) * g.K + k0 + kk, r1 - k0 - kk, wv);
      else b.zero();
    } else if constexpr (KIND == kInput) {
      if (k0 + rr < r1) b.load(W, (k0 + rr) * g.K + n0 + rc, cols - n0 - rc, wv);
      else b.zero();
    } else {
      const int64_t x = k0 + rr < r1 ? x_row(g, k0 + rr) : -1;
      if (x >= 0) b.load(g.X, x * g.xs + n0 + rc, cols - n0 - rc, xv);
      else b.zero();
    }
    __syncthreads();                         // the last round's fragments are read
    if constexpr (KIND == kWeight) {
#pragma unroll
      for (int i = 0; i < 8; ++i) As[(rc + i) * PITCH + rr] = a.v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) As[kr * PITCH + kk + i] = a.v[i];
    }
    if constexpr (KIND == kForward) {
#pragma unroll
      for (int i = 0; i < 8; ++i) Bs[kr * PITCH + kk + i] = b.v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) Bs[(rc + i) * PITCH + rr] = b.v[i];
    }
    __syncthreads();
    const LT* Ar = As + (32 * wm + rl) * PITCH;
    const LT* Br = Bs + (32 * wn + rl) * PITCH;
    if constexpr (TY == kEltF32) {
#pragma unroll
      for (int s = 0; s < KT / 2; ++s)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(Ar[2 * s + kg], Br[2 * s + kg], acc, 0, 0, 0);
    } else {
#pragma unroll
      for (int s = 0; s < KT / 16; ++s) {
        if constexpr (TY == kEltBF16)
          acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              *reinterpret_cast<const bf16x8*>(Ar + 16 * s + 8 * kg),
              *reinterpret_cast<const bf16x8*>(Br + 16 * s + 8 * kg), acc, 0, 0, 0);
        else
          acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(
              *reinterpret_cast<const f16x8*>(Ar + 16 * s + 8 * kg),
              *reinterpret_cast<const f16x8*>(Br + 16 * s + 8 * kg), acc, 0, 0, 0);
      }
    }
  }

  const int c = n0 + 32 * wn + rl;
  if (c >= cols) return;
  const float bias = KIND == kForward && g.b && e < g.E ? g.b[(int64_t)e * g.N + c] : 0.f;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int64_t r = row0 + 32 * wm + 8 * (v >> 2) + 4 * kg + (v & 3);
    if (r >= end) continue;
    float x = acc[v];
    if constexpr (KIND == kWeight) {
      g.dW[we + r * g.K + c] = x;
    } else {
      if constexpr (KIND == kForward) {
        x += bias;
        if (g.relu) x = x > 0.f ? x : 0.f;
      } else if (g.relu && e < g.E) {
        const int64_t xr = x_row(g, r);
        if (!(xr >= 0 && rows::load1<TY>(g.X, xr * g.xs + c) > 0.f)) x = 0.f;
      }
      rows::store1<TY>(g.Y, r * g.ys + c, x);
    }
  }
}

// A value that is the same in the whole wave, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Row tiles that the experts (and the positions of none) need.
template <int BM>
__device__ __forceinline__ int64_t count_tiles(const Product& g) {
  const int lane = threadIdx.x & 63;
  int tiles = 0;
  for (int e = lane; e <= g.E; e += 64) {
    int64_t lo, hi;
    bounds_of(g, e, &lo, &hi);
    tiles += (int)((hi - lo + BM - 1) / BM);
  }
  for (int d = 1; d < 64; d <<= 1) tiles += __shfl_xor(tiles, d);
  return tiles;
}

// The weight gradient's reduction is cut into slices of g.slice positions, so that an expert
// with many rows is many blocks' work: expert e has max(1, ceil(rows / slice)) of them.  One
// slice writes dW itself; the sums of several go to g.part, in order, and are added after.
struct Slice {
  int expert, count;            // slices of this expert
  int64_t lo, hi, partial;      // its positions; place among the partial sums, or -1
};
__device__ __forceinline__ int slices_of(const Product& g, int e, int64_t* lo, int64_t* hi) {
  bounds_of(g, e, lo, hi);
  const int c = (int)((*hi - *lo + g.slice - 1) / g.slice);
  return c > 1 ? c : 1;
}
__device__ __forceinline__ int64_t count_slices(const Product& g) {
  const int lane = threadIdx.x & 63;
  int c = 0;
  for (int e = lane; e < g.E; e += 64) {
    int64_t lo, hi;
    c += slices_of(g, e, &lo, &hi);
  }
  for (int d = 1; d < 64; d <<= 1) c += __shfl_xor(c, d);
  return c;
}
// Slice `unit` of all, or (expert >= 0) the first of that expert.
__device__ __forceinline__ bool find_slice(const Product& g, int64_t unit, int expert, Slice* u) {
  const int lane = threadIdx.x & 63;
  int64_t run = 0, partials = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    const int e = e0 + lane;
    int64_t lo = 0, hi = 0;
    const int c = e < g.E ? slices_of(g, e, &lo, &hi) : 0;
    const int m = c > 1 ? c : 0;
    int upto = c, mupto = m;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d), x = __shfl_up(mupto, d);
      if (lane >= d) {
        upto += v;
        mupto += x;
      }
    }
    const uint64_t hit = expert >= 0 ? __ballot(e == expert) : __ballot(run + upto > unit);
    if (hit) {
      const int at = __ffsll((unsigned long long)hit) - 1;
      const int64_t i = expert >= 0 ? 0 : unit - run - __shfl(upto - c, at);
      const int64_t first = __shfl(lo, at), last = __shfl(hi, at);
      u->expert = e0 + at;
      u->count = __shfl(c, at);
      u->lo = first + i * g.slice;
      u->hi = last < u->lo + g.slice ? last : u->lo + g.slice;
      u->partial = u->count > 1 ? partials + __shfl(mupto - m, at) + i : -1;
      return true;
    }
    run += __shfl(upto, 63);
    partials += __shfl(mupto, 63);
  }
  return false;
}

// What a tile costs beside its rounds of 64 (its first loads, its stores), in rounds.
constexpr int64_t kTileCost = 10;
// The first of the weight gradient's tiles (units in order, `tiles` each) that belongs to the
// last (8 - x) eighths of their cost.
__device__ __forceinline__ int64_t first_by_cost(const Product& g, int tiles, int x) {
  const int lane = threadIdx.x & 63;
  const int64_t full = g.slice / 64 + kTileCost;               // of a whole slice's tile
  auto cost = [&](int64_t rows, int c) {
    return c > 0 ? (c - 1) * full + (rows - (c - 1) * g.slice + 63) / 64 + kTileCost : 0;
  };
  int64_t total = 0;
  for (int e = lane; e < g.E; e += 64) {
    int64_t lo, hi;
    const int c = slices_of(g, e, &lo, &hi);
    total += cost(hi - lo, c);
  }
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  const int64_t target = total * tiles * x / kXcds;
  int64_t run = 0, units = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int64_t lo = 0, hi = 0;
    const int c = e0 + lane < g.E ? slices_of(g, e0 + lane, &lo, &hi) : 0;
    const int64_t mine = cost(hi - lo, c) * tiles;
    int64_t upto = mine;
    int cupto = c;
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t v = __shfl_up(upto, d);
      const int y = __shfl_up(cupto, d);
      if (lane >= d) {
        upto += v;
        cupto += y;
      }
    }
    const uint64_t past = __ballot(run + upto > target);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      int64_t left = target - run - __shfl(upto - mine, at);
      const int64_t rows = __shfl(hi - lo, at);
      const int count = __shfl(c, at);
      int64_t i = left / (full * tiles);
      i = i < count - 1 ? i : count - 1;
      left -= i * full * tiles;
      const int64_t each = i < count - 1 ? full : cost(rows - i * g.slice, 1);
      int64_t t = (left + each - 1) / each;
      t = t < tiles ? t : tiles;
      return (units + __shfl(cupto - c, at) + i) * tiles + t;
    }
    run += __shfl(upto, 63);
    units += __shfl(cupto, 63);
  }
  return units * tiles;
}

// The block's first tile and the end of its XCD's part of all tiles: blocks go to the 8 XCDs in
// turn, and each XCD, which has an L2 of its own, has a run of neighbouring tiles that share
// operands.
template <int KIND, int BM>
__device__ __forceinline__ void part_of(const Product& g, int64_t* first, int64_t* last) {
  const int x = blockIdx.x % kXcds;
  if constexpr (KIND == kWeight) {
    const int tiles = g.row_tiles * g.col_tiles;
    *first = first_by_cost(g, tiles, x);
    *last = x + 1 < (int)kXcds ? first_by_cost(g, tiles, x + 1) : count_slices(g) * tiles;
  } else {
    const int64_t total = count_tiles<BM>(g) * g.col_tiles;
    *first = total * x / kXcds;
    *last = total * (x + 1) / kXcds;
  }
  *first = uniform(*first) + blockIdx.x / kXcds;
  *last = uniform(*last);
}

// dW of the experts with several slices: their partial sums added in order.  A block has
// kJoin elements of one expert.
constexpr int kJoin = 8192;
__global__ __launch_bounds__(kThreads) void join_kernel(Product g) {
  const int64_t count = (int64_t)g.N * g.K;
  const int64_t each = (count + kJoin - 1) / kJoin;
  const int e = (int)(blockIdx.x / each);
  Slice u;
  if (!find_slice(g, 0, e, &u) || u.count < 2) return;
  const float* part = g.part + u.partial * count;
  float* out = g.dW + e * count;
  const int64_t begin = (blockIdx.x % each) * kJoin;
  const int64_t end = count < begin + kJoin ? count : begin + kJoin;
  for (int64_t i = begin + threadIdx.x * 4; i < end; i += kThreads * 4) {   // count % 4 == 0
    float4 s = *reinterpret_cast<const float4*>(part + i);
    for (int z = 1; z < u.count; ++z) {
      const float4 x = *reinterpret_cast<const float4*>(part + z * count + i);
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    *reinterpret_cast<float4*>(out + i) = s;
  }
}

// The 16-bit values of h where those of m are positive, else zero.
template <int TY>
__device__ __forceinline__ uint32_t keep_positive(uint32_t h, uint32_t m) {
  return (half_lo<TY>(m) > 0.f ? h & 0xFFFFu : 0u) | (half_hi<TY>(m) > 0.f ? h & 0xFFFF0000u : 0u);
}

// ------------------------------------------------------------------ 16-bit operands, staged
// The products of 16-bit operands in 16-byte pieces (widths and strides multiples of 8,
// 16-byte aligned arrays).  A block has a BM x BN output tile and a wave a WM x WN part of it
// in 32 x 32 matrix-core tiles.  The reduction advances in rounds of 64 values, so that a row
// is read 128 bytes at a time (half of that costs the first-level cache twice the requests,
// and the forward product 729 us instead of ... at 65536 x 2208 x 2048).  Tiles go from
// memory to LDS directly (one 16-byte load a lane, 1 KB a wave, no registers in between); the
// loads' own bounds check gives zeros for rows and reduction values that are not there.
//
// LDS is a ring of five slots of one operand's round, in the order A0 B0 A1 B1 ...: while
// round j is read, B of round j + 1 and A of round j + 2 are on their way.  A round has two
// half steps, and a half step two parts: one that moves data (the wave's fragments from LDS
// to registers, its share of the loads of one operand) and one that computes (16 matrix-core
// instructions a wave in 256 x 256 tiles).  With eight waves, two on each SIMD, the second
// four run one part behind the first: while one of a SIMD's waves computes the other moves
// data.  Barriers end both parts.  With four waves there are two blocks a compute unit, which
// interleave by themselves, and one barrier a half step.
//
// An operand lies in LDS in one of two forms; the banks serve 256 bytes at a time:
//   by rows (64 reduction values of one row, 128 bytes): a fragment is one 16-byte read of 32
//     rows.  The 16-byte piece c of row r is at c ^ (r / 2 & 7), so that sixteen lanes that
//     read piece c of sixteen rows touch all banks.
//   by reduction (BM or BN values of one reduction index): a fragment is two transposing
//     reads, each giving a lane four reduction values of its row.  32 lanes read 64 bytes of
//     four reduction rows; piece c of reduction row q is at c ^ (4 (q & 3)), which spreads
//     the four over the banks.
// The matrix cores take the columns as their rows: a lane then holds four neighbouring
// columns of one output row, stored together.
//
// Blocks stay: each takes tiles of its XCD's part until there are none.  The parts have equal
// cost, which for the weight gradient, whose tiles are as long as their expert has rows, is
// not equal numbers.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kRound = 64, kHalf = 32;         // reduction values
// An offset past every buffer: reads zeros, writes nothing.  Offsets are below 2^31, and so is
// what is added to them for all lanes, so that the sum never wraps; gathered rows, to which
// nothing is added, reach further.
constexpr uint32_t kNowhere = 0x80000000u, kFar = 0xFFFFFFF0u;

template <int TY>
__device__ __forceinline__ f32x16 mma(s16x8 a, s16x8 b, f32x16 c) {
  if constexpr (TY == kEltBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 16 bytes a lane from base + off + more to lds + 16 * lane (base, more and lds the same in the
// whole wave).
template <uint32_t END = kNowhere>
__device__ __forceinline__ void to_lds(const void* base, uint32_t off, uint32_t more,
                                       uint16_t* lds) {
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)END, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16,
                                           (int)off, (int)more, 0, 0);
}

// 16 bytes a lane from base + off (base the same in the whole wave).
__device__ __forceinline__ uint4 load16(const void* base, uint32_t off) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void*>(base), (short)0, (int)kFar, 0x00020000);
  const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// 16 bytes a lane to base + off (base the same in the whole wave).  No part of the address is
// in the instruction's scalar offset: with one the compiler lets the next instruction write the
// registers that are stored, and the store has been seen to take what that writes.
__device__ __forceinline__ void store16(void* base, uint32_t off, uint4 x) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc(base, (short)0, (int)kNowhere, 0x00020000);
  const u32x4 v = {x.x, x.y, x.z, x.w};
  __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, 0);
}

// Ends a part: the wave's LDS reads are done and at most LOADS of its loads are in flight, in
// every wave (LOADS < 0: any number).
template <int LOADS>
__device__ __forceinline__ void arrive() {
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (LOADS < 0)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LOADS) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void arrive_only() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// ORDER: the weight gradient reads X's rows through g.order.
template <int TY, int KIND, int BM, int BN, int WM, int WN, bool ORDER>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, 2) void wide_kernel(Product g) {
  constexpr int WAVES = (BM / WM) * (BN / WN), WN_WAVES = BN / WN;
  constexpr bool AROW = KIND != kWeight, BROW = KIND == kForward, PAIRED = WAVES == 8;
  constexpr int TI = WM / 32, TJ = WN / 32;
  constexpr int AL = BM * kRound / 512 / WAVES, BL = BN * kRound / 512 / WAVES;
  constexpr int STORES = TI * (KIND == kWeight ? WN / 8 : WN / 16);
  constexpr int SLOT = (BM > BN ? BM : BN) * kRound;           // a ring slot holds either operand
  __shared__ __attribute__((aligned(16))) uint16_t R0[SLOT], R1[SLOT], R2[SLOT], R3[SLOT], R4[SLOT];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / WN_WAVES, wn = w % WN_WAVES;
  const int rl = lane & 31, kg = lane >> 5;
  const int cols = KIND == kForward ? g.N : g.K;

  // A tile: the first of its rows and columns, the end of the rows, the reduction's range.
  struct Tile {
    int e, n0;
    int64_t row0, end, r0, r1;
    float* dW;
  };
  auto find = [&](int64_t at) {
    Tile n;
    n.r0 = 0;
    n.dW = g.dW;
    if constexpr (KIND == kWeight) {
      const uint32_t tiles = g.row_tiles * g.col_tiles, tile = (uint32_t)at % tiles;
      Slice u;
      u.expert = 0; u.lo = u.hi = 0; u.partial = -1;
      find_slice(g, (uint32_t)at / tiles, -1, &u);
      n.e = u.expert;
      n.r0 = u.lo;
      n.r1 = u.hi;
      const int64_t part = uniform(u.partial);
      n.dW = part >= 0 ? g.part + part * g.N * g.K : g.dW + uniform(n.e) * g.N * g.K;
      n.row0 = (int64_t)(tile / (uint32_t)g.col_tiles) * BM;
      n.n0 = (int)(tile % (uint32_t)g.col_tiles) * BN;
      n.end = g.N;
    } else {
      n.n0 = (int)((uint32_t)at % (uint32_t)g.col_tiles) * BN;
      n.e = g.E; n.row0 = n.end = g.n;
      find_tile<BM>(g, (uint32_t)at / (uint32_t)g.col_tiles, &n.e, &n.row0, &n.end);
      n.r1 = n.e < g.E ? (KIND == kForward ? g.K : g.N) : 0;
    }
    n.e = __builtin_amdgcn_readfirstlane(n.e);
    n.n0 = __builtin_amdgcn_readfirstlane(n.n0);
    n.row0 = uniform(n.row0);
    n.end = uniform(n.end);
    n.r0 = uniform(n.r0);
    n.r1 = uniform(n.r1);
    return n;
  };

  // A load takes 8 rows (by rows) or 512 / WIDE reduction rows (by reduction); load q of wave w
  // is number q * WAVES + w.  Where a lane's 16 bytes are: at `base` of the round, plus the
  // lane's offset, plus a number of rows that is the same in the wave.  By rows lane i has row
  // i / 8 and its piece (i % 8) ^ (row / 2 & 7).
  const uint16_t* abase;
  const uint16_t* bbase;
  int64_t astep, bstep;                                        // elements from round to round
  uint32_t aoff, boff, rowoff[AL];                             // bytes
  int arows, brows;                                            // rows that there are
  constexpr int APER = 512 / BM, BPER = 512 / BN;
  constexpr int ALANES = 64 / APER, BLANES = 64 / BPER;
  const int piece = ((lane & 7) ^ ((4 * w + (lane >> 4)) & 7)) * 8;   // first reduction value
  const int64_t ald = KIND == kForward ? g.xs : g.dys, bld = KIND == kWeight ? g.xs : g.K;
  auto aim = [&](const Tile& n) {
    const uint16_t* W =
        static_cast<const uint16_t*>(g.W) + (int64_t)(n.e < g.E ? n.e : 0) * g.N * g.K;
    arows = (int)(n.end - n.row0 < BM ? n.end - n.row0 : BM);
    brows = cols - n.n0 < BN ? cols - n.n0 : BN;
    if constexpr (KIND == kForward) {
      abase = static_cast<const uint16_t*>(g.X) + (g.order ? 0 : n.row0 * ald);
      astep = kRound;
#pragma unroll
      for (int q = 0; q < AL; ++q) {
        const int r = 8 * (q * WAVES + w) + (lane >> 3);
        int64_t x = r < arows ? r : -1;
        if (g.order && x >= 0) x = x_row(g, n.row0 + r);
        rowoff[q] = x >= 0 ? (uint32_t)(x * ald + piece) * 2 : kFar;
      }
    } else if constexpr (KIND == kInput) {
      abase = static_cast<const uint16_t*>(g.dY) + n.row0 * ald;
      astep = kRound;
      aoff = (uint32_t)((lane >> 3) * ald + piece) * 2;
    } else {
      abase = static_cast<const uint16_t*>(g.dY) + n.r0 * ald + n.row0;
      astep = kRound * ald;
      const int kr = w * APER + lane / ALANES, c = ((lane % ALANES) ^ (4 * (kr & 3))) * 8;
      aoff = c < arows ? (uint32_t)((lane / ALANES) * ald + c) * 2 : kNowhere;
    }
    if constexpr (BROW) {
      bbase = W + (int64_t)n.n0 * bld;
      bstep = kRound;
      boff = (uint32_t)((lane >> 3) * bld + piece) * 2;
    } else {
      bbase = (KIND == kInput ? W : static_cast<const uint16_t*>(g.X)) + n.n0;
      bstep = ORDER ? 0 : kRound * bld;
      if (!ORDER) bbase += n.r0 * bld;
      const int kr = w * BPER + lane / BLANES, c = ((lane % BLANES) ^ (4 * (kr & 3))) * 8;
      boff = c < brows ? (uint32_t)((ORDER ? 0 : (lane / BLANES) * bld) + c) * 2 : kNowhere;
    }
  };
  // with ORDER: the slots of the round after the last loaded one, ahead of their use
  // (scalar loads, which do not stand in line with the operands' loads)
  int32_t slot[BL];
  auto fetch_slots = [&](int64_t k) {
    if constexpr (ORDER) {
      const auto* o = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)g.order;
      const int n1 = (int)g.n - 1;
#pragma unroll
      for (int q = 0; q < BL; ++q) {
        const int p = (int)k + (q * WAVES + w) * BPER;         // past the end: any slot, unused
        int32_t v[BPER], i = 0;
#pragma unroll
        for (int j = 0; j < BPER; ++j) v[j] = o[p + j < n1 ? p + j : n1];
#pragma unroll
        for (int j = 0; j < BPER; ++j) i = lane / BLANES == j ? v[j] : i;
        slot[q] = i;
      }
    }
  };

  // Load the next round of an operand, reduction values [k, k + 64).
  auto load_a = [&](uint16_t* A, int64_t k, int64_t r1) {
    const int left = (int)(r1 - k < kRound ? r1 - k : kRound);
#pragma unroll
    for (int q = 0; q < AL; ++q) {
      const int i = q * WAVES + w;
      if constexpr (KIND == kForward) {
        to_lds<kFar>(abase, piece < left ? rowoff[q] : kFar, 0, A + i * 512);
      } else if constexpr (KIND == kInput) {
        const bool in = piece < left && (lane >> 3) < arows - 8 * i;
        to_lds(abase, in ? aoff : kNowhere, (uint32_t)(8 * i * ald) * 2, A + i * 512);
      } else {
        const bool in = lane / ALANES < left - i * APER;
        to_lds(abase, in ? aoff : kNowhere, (uint32_t)(i * APER * ald) * 2, A + i * 512);
      }
    }
    abase += astep;
  };
  auto load_b = [&](uint16_t* B, int64_t k, int64_t r1) {
    const int left = (int)(r1 - k < kRound ? r1 - k : kRound);
#pragma unroll
    for (int q = 0; q < BL; ++q) {
      const int i = q * WAVES + w;
      if constexpr (BROW) {
        const bool in = piece < left && (lane >> 3) < brows - 8 * i;
        to_lds(bbase, in ? boff : kNowhere, (uint32_t)(8 * i * bld) * 2, B + i * 512);
      } else {
        bool in = lane / BLANES < left - i * BPER;
        if constexpr (ORDER) {
          const int32_t x = token_of(g, slot[q]);
          in = in && x >= 0 && boff != kNowhere;
          to_lds<kFar>(bbase, in ? boff + (uint32_t)x * (uint32_t)bld * 2 : kFar, 0, B + i * 512);
        } else {
          to_lds(bbase, in ? boff : kNowhere, (uint32_t)(i * BPER * bld) * 2, B + i * 512);
        }
      }
    }
    bbase += bstep;
    fetch_slots(k + kRound);
  };
  // The first loads of a tile: A0, B0 and A1.
  auto start = [&](const Tile& n) {
    if (n.r1 <= n.r0) return;
    fetch_slots(n.r0);
    load_a(R0, n.r0, n.r1);
    load_b(R1, n.r0, n.r1);
    load_a(R2, n.r0 + kRound, n.r1);
  };

  // Where a lane's fragments are in a slot, in bytes: those of the operand's 32-row tile i and
  // the reduction values 16 s + 8 kg .. + 8 are at `at` with a few bits flipped, plus a constant.
  // (By reduction: the 16 lanes of a group have reduction row + (lane & 15) / 4 and columns
  // 4 (lane & 3) ..)
  auto frag_at = [&](int row, bool byrow, int wide) -> uint32_t {
    if (byrow) return (row + rl) * kRound * 2 + ((kg ^ (rl >> 1 & 7)) * 16);
    const int kr = 8 * kg + ((lane & 15) >> 2);
    const int c = row + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    return kr * wide * 2 + ((c >> 3) ^ (4 * (kr & 3))) * 16 + (c & 7) * 2;
  };
  const uint32_t afrag = frag_at(WM * wm, AROW, BM), bfrag = frag_at(WN * wn, BROW, BN);
  auto frag = [&](const uint16_t* L, uint32_t at, int i, int s, auto byrow, auto wide) -> s16x8 {
    const char* p = reinterpret_cast<const char*>(L);
    if constexpr (decltype(byrow)::value) {
      return *reinterpret_cast<const s16x8*>(p + (at ^ (32 * s)) + 32 * i * kRound * 2);
    } else {
      constexpr int WIDE = decltype(wide)::value;
      typedef __attribute__((address_space(3))) s16x4* P;
      p += (at ^ (64 * i)) + 16 * s * WIDE * 2;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 4 * WIDE * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  };

  f32x16 acc[TI][TJ];
  // Half step h of a round: `ahead` issues its loads and arrives.
  auto half = [&](const uint16_t* A, const uint16_t* B, auto h, auto ahead) {
    s16x8 a[2][TI], b[2][TJ];
    // the addresses are made here each time: kept for all slots they would take the registers
    // that the accumulators need
    uint32_t aat = afrag, bat = bfrag;
    asm volatile("" : "+v"(aat), "+v"(bat));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        b[s][j] = frag(B, bat, j, 2 * decltype(h)::value + s,
                       std::integral_constant<bool, BROW>{}, std::integral_constant<int, BN>{});
#pragma unroll
      for (int i = 0; i < TI; ++i)
        a[s][i] = frag(A, aat, i, 2 * decltype(h)::value + s,
                       std::integral_constant<bool, AROW>{}, std::integral_constant<int, BM>{});
    }
    ahead();
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = mma<TY>(b[s][j], a[s][i], acc[i][j]);
    __builtin_amdgcn_s_setprio(0);
    if constexpr (PAIRED) arrive_only();
  };

  // The tile whose first loads are on their way: its sums into acc.  `stores`: of the tile
  // before, issued after the loads.
  auto multiply = [&](const Tile& n, bool stores) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int64_t r0 = n.r0, r1 = n.r1;
    const int halves = (int)((r1 - r0 + kHalf - 1) / kHalf), rounds = (halves + 1) >> 1;
    if (halves <= 0) return;
    // (Loads past the last round read nowhere: the counts of loads in flight stay the same, and
  // all have ended when the last half step does.)
  // Round j on A and B; Bn takes B of round j + 1 (its slot held A of round j - 1), An takes A
    // of round j + 2 (its slot held B of round j - 1).
    auto round = [&](const uint16_t* A, const uint16_t* B, uint16_t* Bn, uint16_t* An, int j) {
      half(A, B, std::integral_constant<int, 0>{}, [&] {
        load_b(Bn, r0 + (int64_t)(j + 1) * kRound, r1);
        if (2 * j + 1 < halves) arrive<-1>();
        else arrive<0>();
      });
      if (2 * j + 1 < halves)
        half(A, B, std::integral_constant<int, 1>{}, [&] {
          // round j + 1 has landed when at most A of round j + 2 is in flight
          load_a(An, r0 + (int64_t)(j + 2) * kRound, r1);
          if (j + 1 < rounds) arrive<AL>();
          else arrive<0>();
        });
    };

    // A0 and B0 have landed when at most A1 and the stores after it are in flight
    if (stores) arrive<AL + STORES>();
    else arrive<AL>();
    if (PAIRED && w >= WAVES / 2) arrive_only();
    for (int j = 0; j < rounds; j += 5) {
      round(R0, R1, R3, R4, j);
      if (j + 1 < rounds) round(R2, R3, R0, R1, j + 1);
      if (j + 2 < rounds) round(R4, R0, R2, R3, j + 2);
      if (j + 3 < rounds) round(R1, R2, R4, R0, j + 3);
      if (j + 4 < rounds) round(R3, R4, R1, R2, j + 4);
    }
    if (PAIRED && w < WAVES / 2) arrive_only();
  };

  // acc[i][j][v] is row 32 i + rl, column 32 j + 8 (v / 4) + 4 kg + v % 4 of the wave's part.
  // 32 rows at a time go through 8 KB of LDS a wave (of the two slots that `start` leaves
  // free), so that a store is whole 16-byte pieces along rows.  Every store is issued, those
  // outside the tile to nowhere: `multiply` counts them.
  constexpr int EACH = SLOT * 2 / 8192;                        // waves a slot holds
  static_assert(2 * EACH >= WAVES, "the waves' parts fit");
  char* const out = reinterpret_cast<char*>(w < EACH ? R3 : R4) + (w % EACH) * 8192;
  auto finish = [&](const Tile& n, const f32x4 (&bias)[TJ][4]) {
    constexpr int SIZE = KIND == kWeight ? 4 : 2, PIECE = 16 / SIZE, LR = WN / PIECE;
    const int64_t ld = KIND == kWeight ? g.K : g.ys;
    const int64_t rw = n.row0 + WM * wm;                       // the wave's first row
    const int cw = n.n0 + WN * wn;                             // and column
    char* base = KIND == kWeight ? reinterpret_cast<char*>(n.dW) : static_cast<char*>(g.Y);
    base += (rw * ld + cw) * SIZE;
    // this lane's row and column in the 64 / LR rows of a store (from a lane number that the
    // compiler does not know: what it made of it would stay in registers over the products)
    int me = lane;
    asm volatile("" : "+v"(me));
    const int l = me % LR, rr = me / LR, rl = me & 31, kg = me >> 5;
    const bool in = cw + l * PIECE < cols;
    const int rows = (int)(n.end - rw < WM ? n.end - rw : WM);
    const uint32_t off = (uint32_t)(rr * ld + l * PIECE) * SIZE;
    // with x_relu: the input's values at the same places
    const bool masked = KIND == kInput && g.relu && n.e < g.E;
    const uint16_t* xbase = static_cast<const uint16_t*>(g.X) + cw + (g.order ? 0 : rw * g.xs);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = 32 * j + 8 * q + 4 * kg;
          float x[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            x[v] = acc[i][j][4 * q + v];
            if constexpr (KIND == kForward) {
              x[v] += bias[j][q][v];
              if (g.relu) x[v] = x[v] > 0.f ? x[v] : 0.f;
            }
          }
          if constexpr (KIND == kWeight) {
            *reinterpret_cast<float4*>(out + rl * WN * 4 + ((c >> 2) ^ (rl & 15)) * 16) =
                make_float4(x[0], x[1], x[2], x[3]);
          } else {
            uint2 h;
            h.x = to_half<TY, false>(x[0], 0u) | (to_half<TY, false>(x[1], 0u) << 16);
            h.y = to_half<TY, false>(x[2], 0u) | (to_half<TY, false>(x[3], 0u) << 16);
            *reinterpret_cast<uint2*>(out + rl * (WN + 8) * 2 + c * 2) = h;
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int t = 0; t < 32 * LR / 64; ++t) {
        const int r = t * (64 / LR) + rr;                      // of the 32 staged rows
        const bool here = in && 32 * i + r < rows;
        uint4 h;
        if constexpr (KIND == kWeight)
          h = *reinterpret_cast<const uint4*>(out + r * WN * 4 + (l ^ (r & 15)) * 16);
        else
          h = *reinterpret_cast<const uint4*>(out + r * (WN + 8) * 2 + l * 16);
        if constexpr (KIND == kInput) {
          if (masked) {
            int32_t x = 32 * i + r;
            if (g.order) x = here ? token_of(g, g.order[rw + x]) : -1;
            const uint32_t from = ((uint32_t)x * (uint32_t)g.xs + l * PIECE) * 2;
            const uint4 m = load16(xbase, here && x >= 0 ? from : kFar);
            h.x = keep_positive<TY>(h.x, m.x);
            h.y = keep_positive<TY>(h.y, m.y);
            h.z = keep_positive<TY>(h.z, m.z);
            h.w = keep_positive<TY>(h.w, m.w);
          }
        }
        const uint32_t more = (uint32_t)((32 * i + t * (64 / LR)) * ld) * SIZE;
        store16(base, here ? off + more : kNowhere, h);
      }
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // The next tile's first loads are issued before this tile's results are stored.
  int64_t at, last;
  const int64_t stride = gridDim.x / kXcds;
  part_of<KIND, BM>(g, &at, &last);
  if (at >= last) return;
  Tile n = find(at);
  aim(n);
  start(n);
  for (bool stores = false;; stores = true) {
    multiply(n, stores);
    f32x4 bias[TJ][4];
    if constexpr (KIND == kForward) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = n.n0 + WN * wn + 32 * j + 8 * q + 4 * kg;
          const bool in = g.b && n.e < g.E && c < cols;
#pragma unroll
          for (int v = 0; v < 4; ++v) bias[j][q][v] = in ? g.b[(int64_t)n.e * g.N + c + v] : 0.f;
        }
    }
    const Tile done = n;
    at += stride;
    if (at < last) {
      n = find(at);
      aim(n);
      start(n);
    }
    finish(done, bias);
    if (at >= last) break;
  }
}

// db[e, c] = sum of dY over the expert's rows.  Like the weight gradient's reduction it is cut
// into slices (of g.slice rows here), which write db itself or, where an expert has several,
// partial sums [unit, N] that bias_join_kernel adds in order.  A block has one slice and
// LR lanes along the columns, VW columns each, times 256 / LR rows, four of them in flight.  Bound by reading dY once.
template <int TY, int VW>
__global__ __launch_bounds__(kThreads) void bias_grad_kernel(Product g, int LR,
                                                             float* __restrict__ db) {
  __shared__ float red[kThreads * VW];
  const int t = threadIdx.x, l = t & (LR - 1), r = t / LR, R = kThreads / LR;
  const int c = ((int)(blockIdx.x % g.col_tiles) * LR + l) * VW;
  Slice u;
  if (!find_slice(g, blockIdx.x / g.col_tiles, -1, &u)) return;
  float s[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) s[e] = 0.f;
  using P = rows::Piece<TY, (VW > 1)>;
  if (c < g.N) {
    int64_t p = u.lo + r;
    for (; p + 3 * R < u.hi; p += 4 * R) {
      P x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i].load(g.dY, (p + i * R) * g.dys + c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e) s[e] += x[i].v[e];
    }
    for (; p < u.hi; p += R) {
      P x;
      x.load(g.dY, p * g.dys + c);
#pragma unroll
      for (int e = 0; e < VW; ++e) s[e] += x.v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < VW; ++e) red[t * VW + e] = s[e];
  for (int d = kThreads / 2; d >= LR; d >>= 1) {
    __syncthreads();
    if (t < d)
#pragma unroll
      for (int e = 0; e < VW; ++e) red[t * VW + e] += red[(t + d) * VW + e];
  }
  if (t >= LR || c >= g.N) return;
  float* out = u.partial >= 0 ? g.part + u.partial * g.N : db + (int64_t)u.expert * g.N;
#pragma unroll
  for (int e = 0; e < VW; ++e) out[c + e] = red[t * VW + e];
}

__global__ __launch_bounds__(kThreads) void bias_join_kernel(Product g, float* __restrict__ db) {
  const int e = (int)(blockIdx.x / g.col_tiles);
  const int c = (int)(blockIdx.x % g.col_tiles) * kThreads + threadIdx.x;
  Slice u;
  if (!find_slice(g, 0, e, &u) || u.count < 2 || c >= g.N) return;
  const float* part = g.part + u.partial * g.N + c;
  float s = part[0];
  for (int z = 1; z < u.count; ++z) s += part[(int64_t)z * g.N];
  db[(int64_t)e * g.N + c] = s;
}

}  // namespace experts

static experts::Product expert_product(const void* X, int64_t xs, int64_t x_rows,
                                       const int32_t* order, int k, const int32_t* offsets,
                                       int64_t n, int E, int K, const void* W, int N) {
  experts::Product g{};
  g.X = X; g.xs = xs; g.x_rows = x_rows; g.order = order;
  // with 2^b >= k: kmul = floor(2^(31 + b) / k) + 1 exceeds the quotient by at most 1, which
  // moves i * kmul / 2^(31 + b) by less than 2^-b <= 1 / k: never past the next integer
  while (((int64_t)1 << g.kshift) < k) ++g.kshift;
  g.kmul = (uint32_t)((((uint64_t)1 << (31 + g.kshift)) / (uint64_t)(k > 0 ? k : 1)) + 1);
  g.offsets = offsets; g.n = n; g.E = E; g.K = K; g.N = N; g.W = W;
  return g;
}

// Row tiles that n rows in E + 1 pieces can need.
static int64_t most_tiles(int64_t n, int E, int BM) { return n / BM + E + 1; }

// Whether a product takes the staged 16-bit kernel: everything in whole 16-byte pieces, and a
// block's rows within 32-bit byte offsets of its first (of X's first, where rows are gathered).
static bool wide_ok(const experts::Product& g, int dtype) {
  auto ok = [](const void* p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride % 8 == 0 &&
           stride < ((int64_t)1 << 21);          // 256 rows: 2^30 bytes
  };
  if (dtype == kEltF32 || g.K % 8 || g.N % 8) return false;
  if (!ok(g.X, g.xs) || !ok(g.W, g.K) || !ok(g.Y, g.ys) || !ok(g.dY, g.dys)) return false;
  return !g.order || g.x_rows * g.xs < ((int64_t)1 << 31) - ((int64_t)1 << 20);
}

template <int TY, int KIND, int BM, int BN, int WM, int WN>
static hipError_t launch_wide(experts::Product g, hipStream_t s) {
  const int cols = KIND == experts::kForward ? g.N : g.K;
  g.col_tiles = (cols + BN - 1) / BN;
  g.row_tiles = (g.N + BM - 1) / BM;
  const int64_t blocks = KIND == experts::kWeight
                             ? (g.n / g.slice + g.E) * (int64_t)g.row_tiles * g.col_tiles
                             : most_tiles(g.n, g.E, BM) * g.col_tiles;
  // as many blocks as run at once, or the tiles there can be
  int64_t most = 256 * (BM == 256 ? 1 : 2);
  if (getenv("CTR_NOSTAY") && KIND != experts::kWeight) most = 1 << 30;
  const int64_t grid = (blocks < most ? blocks : most) + kXcds - 1;
  const unsigned whole = (unsigned)(grid / kXcds * kXcds), threads = (BM / WM) * (BN / WN) * 64;
  if (KIND == experts::kWeight && g.order)
    experts::wide_kernel<TY, KIND, BM, BN, WM, WN, KIND == experts::kWeight>
        <<<whole, threads, 0, s>>>(g);
  else
    experts::wide_kernel<TY, KIND, BM, BN, WM, WN, false><<<whole, threads, 0, s>>>(g);
  return hipGetLastError();
}

// 256 x 256 tiles, or 128 x 128 where the larger ones are too few to fill the chip.
static bool big_tiles(int64_t row_tiles, int cols) {
  return row_tiles * ((cols + 255) / 256) >= 512;
}

template <int TY, int KIND>
static hipError_t launch_product(experts::Product g, bool wide, hipStream_t s) {
  if constexpr (TY != kEltF32) {
    if (wide) {
      const int v = getenv("CTR_TILE") ? atoi(getenv("CTR_TILE")) : 0;
      if (v == 0) return launch_wide<TY, KIND, 256, 256, 128, 64>(g, s);
      if (v == 1) return launch_wide<TY, KIND, 256, 128, 64, 64>(g, s);
      return launch_wide<TY, KIND, 128, 128, 64, 64>(g, s);
    }
  }
  const int cols = KIND == experts::kForward ? g.N : g.K;
  g.col_tiles = (cols + 63) / 64;
  g.row_tiles = (g.N + 63) / 64;
  const int64_t rows = KIND == experts::kWeight ? (int64_t)g.E * g.row_tiles
                                                : most_tiles(g.n, g.E, 64);
  experts::product_kernel<TY, KIND>
      <<<(unsigned)(rows * g.col_tiles), experts::kThreads, 0, s>>>(g);
  return hipGetLastError();
}

// Positions a slice of the weight gradient's reduction: about four blocks a compute unit in
// all, at least 512.
static void set_slices(experts::Product& g) {
  const int64_t big = (int64_t)((g.N + 255) / 256) * ((g.K + 255) / 256);
  const int64_t small = (int64_t)((g.N + 127) / 128) * ((g.K + 127) / 128);
  g.slice_big = big * g.E >= 512;
  const int64_t tiles = g.slice_big ? big : small;
  int64_t slice = (g.n * tiles + 1023) / 1024;
  slice = slice < 512 ? 512 : slice;
  if (getenv("CTR_SLICE")) slice = atoi(getenv("CTR_SLICE"));
  g.slice = (slice + 63) / 64 * 64;
}

static int64_t most_partials(const experts::Product& g) {
  // experts with several slices have more than `slice` rows each
  const int64_t a = 2 * (g.n / g.slice), b = g.n / g.slice + g.E;
  return a < b ? a : b;
}

hipError_t launch_expert_dense_fwd(const void* X, int dtype, int64_t xs, int64_t x_rows,
                                   const int32_t* order, int k, const int32_t* offsets, int64_t n,
                                   int E, int K, const void* W, const float* b, int N, bool relu,
                                   void* Y, int64_t ys, hipStream_t s) {
  if (n == 0) return hipSuccess;
  experts::Product g = expert_product(X, xs, x_rows, order, k, offsets, n, E, K, W, N);
  g.b = b; g.relu = relu; g.Y = Y; g.ys = ys;
  return by_type(dtype, [&](auto ty) {
    return launch_product<decltype(ty)::value, experts::kForward>(g, wide_ok(g, dtype), s);
  });
}

// Rows a slice of the bias gradient: at least 256, at most about 1024 slices.
static int64_t bias_slice(int64_t n) {
  const int64_t s = (n + 1023) / 1024;
  return s < 256 ? 256 : s;
}

size_t expert_dense_bwd_workspace_bytes(int64_t n, int E, int K, int N, int dtype) {
  experts::Product g = expert_product(nullptr, K, n, nullptr, 1, nullptr, n, E, K, nullptr, N);
  int64_t need = 0;
  if (dtype != kEltF32 && K % 8 == 0 && N % 8 == 0) {
    set_slices(g);
    need = most_partials(g) * N * K;
  }
  // the bias gradient's sums come after the weight gradient's are joined
  g.slice = bias_slice(n);
  const int64_t bias = most_partials(g) * N;
  return (size_t)(need > bias ? need : bias) * sizeof(float) + 256;
}

hipError_t launch_expert_dense_bwd(const void* X, int dtype, int64_t xs, int64_t x_rows,
                                   const int32_t* order, int k, const int32_t* offsets, int64_t n,
                                   int E, int K, const void* W, int N, bool x_relu,
                                   const void* dY, int64_t dys, void* dX, int64_t dxs, float* dW,
                                   float* db, void* workspace, hipStream_t s) {
  experts::Product g = expert_product(X, xs, x_rows, order, k, offsets, n, E, K, W, N);
  g.relu = x_relu; g.dY = dY; g.dys = dys;
  return by_type(dtype, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    hipError_t e = hipSuccess;
    if (dX && n > 0) {
      experts::Product h = g;
      if (!x_relu) {                   // X is not read
        h.X = nullptr; h.xs = 0; h.x_rows = 0; h.order = nullptr;
      }
      h.Y = dX; h.ys = dxs;
      e = launch_product<TY, experts::kInput>(h, wide_ok(h, dtype), s);
    }
    if (e == hipSuccess && dW) {
      experts::Product h = g;
      h.W = nullptr;
      h.dW = dW;
      h.part = static_cast<float*>(workspace);
      set_slices(h);
      const bool wide = wide_ok(h, dtype) && (reinterpret_cast<uintptr_t>(dW) & 15u) == 0;
      e = launch_product<TY, experts::kWeight>(h, wide, s);
      if (e == hipSuccess && wide && n > h.slice) {
        const int64_t each = ((int64_t)N * K + experts::kJoin - 1) / experts::kJoin;
        experts::join_kernel<<<(unsigned)(E * each), experts::kThreads, 0, s>>>(h);
        e = hipGetLastError();
      }
    }
    if (e == hipSuccess && db) {
      g.slice = bias_slice(n);
      g.part = static_cast<float*>(workspace);
      const int VW = TY == kEltF32 ? 4 : 8;
      const bool vec = rows::row_vec(dY, dys, N, TY == kEltF32 ? 4 : 2);
      const int LR = row_lanes(vec ? N / VW : N), wide = LR * (vec ? VW : 1);
      g.col_tiles = (N + wide - 1) / wide;
      const unsigned blocks = (unsigned)((n / g.slice + E) * g.col_tiles);
      if (vec)
        experts::bias_grad_kernel<TY, VW><<<blocks, experts::kThreads, 0, s>>>(g, LR, db);
      else
        experts::bias_grad_kernel<TY, 1><<<blocks, experts::kThreads, 0, s>>>(g, LR, db);
      if (n > g.slice) {
        g.col_tiles = (N + experts::kThreads - 1) / experts::kThreads;
        experts::bias_join_kernel<<<(unsigned)(E * g.col_tiles), experts::kThreads, 0, s>>>(g, db);
      }
      e = hipGetLastError();
    }
    return e;
  });
}

}  // namespace ctr

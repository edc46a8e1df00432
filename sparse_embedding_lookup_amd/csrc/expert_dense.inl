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
namespace ctr {
namespace experts {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;

struct Product {
  const void* X;
  int64_t xs, x_rows;
  const int32_t* order;         // nullable: positions are X's rows
  int k;
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
  float* dW;                    // dW, or its partial sums
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

// Row of X that position p reads, or -1 (a slot outside X: its row reads as zeros).
__device__ __forceinline__ int64_t x_row(const Product& g, int64_t p) {
  if (!g.order) return p < g.x_rows ? p : -1;
  const int64_t i = g.order[p];
  const int64_t r = i >= 0 ? i / g.k : -1;
  return r < g.x_rows ? r : -1;
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

// db[e, c] = sum of dY over the expert's rows: a block has 64 columns of one expert, each of
// its four waves every fourth row; the waves' sums are added in order.
template <int TY>
__global__ __launch_bounds__(kThreads) void bias_grad_kernel(Product g, float* __restrict__ db) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int e = (int)(blockIdx.x / g.col_tiles);
  const int c = (int)(blockIdx.x % g.col_tiles) * 64 + lane;
  int64_t lo, hi;
  bounds_of(g, e, &lo, &hi);
  float s = 0.f;
  if (c < g.N)
    for (int64_t p = lo + w; p < hi; p += 4) s += rows::load1<TY>(g.dY, p * g.dys + c);
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < g.N)
    db[(int64_t)e * g.N + c] = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
}

}  // namespace experts

static experts::Product expert_product(const void* X, int64_t xs, int64_t x_rows,
                                       const int32_t* order, int k, const int32_t* offsets,
                                       int64_t n, int E, int K, const void* W, int N) {
  experts::Product g{};
  g.X = X; g.xs = xs; g.x_rows = x_rows; g.order = order; g.k = k;
  g.offsets = offsets; g.n = n; g.E = E; g.K = K; g.N = N; g.W = W;
  return g;
}

// Row tiles that n rows in E + 1 pieces can need.
static int64_t most_tiles(int64_t n, int E, int BM) { return n / BM + E + 1; }

hipError_t launch_expert_dense_fwd(const void* X, int dtype, int64_t xs, int64_t x_rows,
                                   const int32_t* order, int k, const int32_t* offsets, int64_t n,
                                   int E, int K, const void* W, const float* b, int N, bool relu,
                                   void* Y, int64_t ys, hipStream_t s) {
  if (n == 0) return hipSuccess;
  experts::Product g = expert_product(X, xs, x_rows, order, k, offsets, n, E, K, W, N);
  g.b = b; g.relu = relu; g.Y = Y; g.ys = ys;
  g.col_tiles = (N + 63) / 64;
  const unsigned blocks = (unsigned)(most_tiles(n, E, 64) * g.col_tiles);
  return by_type(dtype, [&](auto ty) {
    experts::product_kernel<decltype(ty)::value, experts::kForward>
        <<<blocks, experts::kThreads, 0, s>>>(g);
    return hipGetLastError();
  });
}

size_t expert_dense_bwd_workspace_bytes(int64_t n, int E, int K, int N, int dtype) { return 256; }

hipError_t launch_expert_dense_bwd(const void* X, int dtype, int64_t xs, int64_t x_rows,
                                   const int32_t* order, int k, const int32_t* offsets, int64_t n,
                                   int E, int K, const void* W, int N, bool x_relu,
                                   const void* dY, int64_t dys, void* dX, int64_t dxs, float* dW,
                                   float* db, void* workspace, hipStream_t s) {
  experts::Product g = expert_product(X, xs, x_rows, order, k, offsets, n, E, K, W, N);
  g.relu = x_relu; g.dY = dY; g.dys = dys; g.Y = dX; g.ys = dxs; g.dW = dW;
  return by_type(dtype, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    if (dX && n > 0) {
      g.col_tiles = (K + 63) / 64;
      const unsigned blocks = (unsigned)(most_tiles(n, E, 64) * g.col_tiles);
      experts::product_kernel<TY, experts::kInput><<<blocks, experts::kThreads, 0, s>>>(g);
    }
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && dW) {
      g.col_tiles = (K + 63) / 64;
      g.row_tiles = (N + 63) / 64;
      const unsigned blocks = (unsigned)((int64_t)E * g.row_tiles * g.col_tiles);
      experts::product_kernel<TY, experts::kWeight><<<blocks, experts::kThreads, 0, s>>>(g);
      e = hipGetLastError();
    }
    if (e == hipSuccess && db) {
      g.col_tiles = (N + 63) / 64;
      const unsigned blocks = (unsigned)((int64_t)E * g.col_tiles);
      experts::bias_grad_kernel<TY><<<blocks, experts::kThreads, 0, s>>>(g, db);
      e = hipGetLastError();
    }
    return e;
  });
}

}  // namespace ctr

// rms_norm.inl -- root-mean-square norm of rows, with the residual's addition before it and the
// result in 8 bits after it, and its gradients; rows in 8 bits by themselves.  Part of the
// translation unit of dense.hip.
//
//   s = x + r (rounded once to the rows' type: the residual stream, which is what is normed)
//   y = s * rstd * w,   rstd = (mean of s^2 + eps)^(-1/2)
//   8 bits: scale = max(largest |y|, 2^-100) / 448,  code = e4m3(y * (448 / max(..)))
//   backward, dn = dy * w:   dx = rstd (dn - s rstd^2 mean(dn s)) + ds,   dw = sum of dy s rstd
//
// A row lies in the registers of G lanes (a power of two up to 64) or of a block of 256, P runs
// of E elements a lane, so that memory is read once; statistics are fp32 sums of the lanes' own
// sums.  Groups stay and take row after row, with the weights in registers.
// Bound by memory: 65536 x 1024 bf16 with the residual's sum written 93 us (5.8 TB/s), backward with
// the other gradient 114 us (4.7 TB/s) and 5 for the weight's partial sums; 16387 x 479 fp32 12, 17
// and 4 us (5.3 and 5.4 TB/s); 48 x 1024 into 8 bits 5.1 us, latency.
namespace ctr {
namespace norm {

constexpr int kThreads = 256;
constexpr float kMost8 = 448.f;                // largest e4m3 value

// The group's sum (or largest bits) in every lane of it: G lanes of a wave, or with BLOCK all
// 256 threads, through `room` (a slot for every call of a row).
template <bool BLOCK>
__device__ __forceinline__ float sum_of(int G, float v, float* room) {
  v = rows::group_sum(BLOCK ? 64 : G, v);
  if constexpr (BLOCK) {
    if ((threadIdx.x & 63) == 0) room[threadIdx.x >> 6] = v;
    __syncthreads();
    v = ((room[0] + room[1]) + room[2]) + room[3];
  }
  return v;
}
template <bool BLOCK>
__device__ __forceinline__ uint32_t most_of(int G, uint32_t v, float* room) {
  rows::butterfly(BLOCK ? 64 : G, [&](auto get) {
    const uint32_t o = (uint32_t)get((int)v);
    v = o > v ? o : v;
  });
  if constexpr (BLOCK) {
    uint32_t* r = reinterpret_cast<uint32_t*>(room);
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = v;
    __syncthreads();
    uint32_t m = r[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) m = r[i] > m ? r[i] : m;
    v = m;
  }
  return v;
}

struct Args {
  const void* X;
  int64_t xs;
  const void* R;                // nullable
  int64_t rs;
  const float* w;               // nullable: 1
  int64_t n;
  int D, G;
  float eps;
  void* S;                      // nullable (without R)
  int64_t ss;
  void* Y;
  int64_t ys;
  float* y_scale;               // 8 bits
  float* rstd;                  // nullable
  // backward
  const void* dY;
  int64_t dys;
  const void* dS;               // nullable
  int64_t dss;
  void* dX;
  int64_t dxs;
  float* part;                  // [blocks, D] partial sums of dw, nullable
};

enum Mode { kPlain = 0, kNorm8 = 1, kRows8 = 2 };

// TY: the rows' type.  kRows8: no norm, no weight, no residual: the rows in 8 bits.
template <int TY, int P, bool BLOCK, int MODE>
__global__ __launch_bounds__(kThreads) void fwd_kernel(Args a) {
  constexpr int E = TY == kEltF32 ? 4 : 8;
  __shared__ float room[2][2][4];
  const int G = BLOCK ? kThreads : a.G, l = threadIdx.x & (G - 1);
  const int64_t step = (int64_t)gridDim.x * (kThreads / G);
  float w[P][E];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = (p * G + l) * E;
    Run<kEltF32, E> x;
    if (MODE != kRows8 && a.w) x.load_some(a.w, c, a.D - c);
#pragma unroll
    for (int e = 0; e < E; ++e) w[p][e] = MODE != kRows8 && a.w ? x.at(e) : 1.f;
  }
  int flip = 0;
  for (int64_t r = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; ; r += step) {
    // a group's lanes, and with BLOCK all threads, leave together
    if (r >= a.n) break;
    Run<TY, E> x[P], y[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + l) * E;
      x[p].load_some(a.X, r * a.xs + c, a.D - c);
      if (MODE != kRows8 && a.R) y[p].load_some(a.R, r * a.rs + c, a.D - c);
    }
    float s[P][E], sum = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + l) * E;
#pragma unroll
      for (int e = 0; e < E; ++e) s[p][e] = x[p].at(e);
      if (MODE != kRows8 && a.R) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          s[p][e] += y[p].at(e);
          if constexpr (TY != kEltF32) s[p][e] = half_lo<TY>(to_half<TY, false>(s[p][e], 0u));
        }
        store_some<TY, E>(a.S, r * a.ss + c, s[p], a.D - c);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sum += s[p][e] * s[p][e];
    }
    if constexpr (MODE != kRows8) {
      sum = sum_of<BLOCK>(G, sum, room[flip][0]);
      const float rstd = 1.f / sqrtf(sum / (float)a.D + a.eps);
      if (a.rstd && l == 0) a.rstd[r] = rstd;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < E; ++e) s[p][e] = s[p][e] * rstd * w[p][e];
    }
    if constexpr (MODE == kPlain) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = (p * G + l) * E;
        store_some<TY, E>(a.Y, r * a.ys + c, s[p], a.D - c);
      }
    } else {
      // the largest magnitude by its bits, in which NaN is above infinity
      uint32_t most = 0u;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t b = __float_as_uint(s[p][e]) & 0x7FFFFFFFu;
          most = b > most ? b : most;
        }
      most = most_of<BLOCK>(G, most, room[flip][1]);
      const float least = 7.888609052210118e-31f;              // 2^-100
      const float top = __uint_as_float(most) < least ? least : __uint_as_float(most);
      const float by = kMost8 / top;
      if (l == 0) a.y_scale[r] = top / kMost8;
      // zeros to the next multiple of 16
      const int width = (a.D + 15) & ~15;
      if (l == 0)
        for (int c = P * G * E; c < width; c += 4)
          *reinterpret_cast<uint32_t*>(static_cast<char*>(a.Y) + r * a.ys + c) = 0u;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = (p * G + l) * E;
        uint32_t u[E / 4];
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          float q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            q[e] = c + 4 * i + e < a.D ? s[p][4 * i + e] * by : 0.f;
            q[e] = q[e] > kMost8 ? kMost8 : q[e] < -kMost8 ? -kMost8 : q[e];
          }
          int o = 0;
          o = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], o, false);
          o = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], o, true);
          u[i] = (uint32_t)o;
        }
        if (c < width)
          __builtin_memcpy(static_cast<char*>(a.Y) + r * a.ys + c, u, sizeof(u));
      }
    }
    flip ^= 1;                                 // slots are written again two barriers later
  }
}

template <int TY, int P, bool BLOCK>
__global__ __launch_bounds__(kThreads) void bwd_kernel(Args a) {
  constexpr int E = TY == kEltF32 ? 4 : 8;
  __shared__ float room[2][4];
  const int G = BLOCK ? kThreads : a.G, l = threadIdx.x & (G - 1);
  const int64_t step = (int64_t)gridDim.x * (kThreads / G);
  float w[P][E], dw[P][E];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = (p * G + l) * E;
    Run<kEltF32, E> x;
    if (a.w) x.load_some(a.w, c, a.D - c);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      w[p][e] = a.w ? x.at(e) : 1.f;
      dw[p][e] = 0.f;
    }
  }
  int flip = 0;
  for (int64_t r = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; r < a.n; r += step) {
    Run<TY, E> x[P], y[P], z[P];
    const float rstd = a.rstd[r];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + l) * E;
      x[p].load_some(a.X, r * a.xs + c, a.D - c);
      y[p].load_some(a.dY, r * a.dys + c, a.D - c);
      if (a.dS) z[p].load_some(a.dS, r * a.dss + c, a.D - c);
    }
    float dot = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float dy = y[p].at(e), s = x[p].at(e);
        dw[p][e] += dy * (s * rstd);
        dot += (dy * w[p][e]) * s;
      }
    dot = sum_of<BLOCK>(G, dot, room[flip]);
    const float back = dot / (float)a.D * rstd * rstd;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + l) * E;
      float d[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        d[e] = rstd * (y[p].at(e) * w[p][e] - x[p].at(e) * back);
        if (a.dS) d[e] += z[p].at(e);
      }
      store_some<TY, E>(a.dX, r * a.dxs + c, d, a.D - c);
    }
    flip ^= 1;
  }
  if (!a.part) return;
  // the block's sum of dw: the groups' in order
  if constexpr (BLOCK) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + l) * E;
      store_some<kEltF32, E>(a.part, (int64_t)blockIdx.x * a.D + c, dw[p], a.D - c);
    }
  } else {
    __shared__ float sums[kThreads * E];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) sums[e * kThreads + threadIdx.x] = dw[p][e];
      __syncthreads();
      const int c = (p * G + l) * E;
      if ((int)threadIdx.x < G && c < a.D) {
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
        for (int u = 0; u < kThreads / G; ++u)
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] += sums[e * kThreads + u * G + l];
        store_some<kEltF32, E>(a.part, (int64_t)blockIdx.x * a.D + c, v, a.D - c);
      }
    }
  }
}

// dw: a block has 16 columns, its 64 groups of 16 lanes every 64th block's partial sums, sixteen in
// flight, joined in order: one trip to memory where 1024 blocks left theirs.  (64 columns a block and
// every sixteenth block's sums a wave 5.6 us for 3.9, four waves with eight in flight 13.)
constexpr int kJoinCols = 16, kJoinThreads = 1024, kJoinWaves = kJoinThreads / 64;
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const float* __restrict__ part,
                                                            int blocks, int D,
                                                            float* __restrict__ dw) {
  __shared__ float sums[kJoinWaves][kJoinCols];
  constexpr int DEEP = 16, GROUPS = kJoinThreads / kJoinCols;
  const int l = threadIdx.x % kJoinCols, c = (int)blockIdx.x * kJoinCols + l;
  float s = 0.f;
  for (int b = threadIdx.x / kJoinCols; b < blocks; b += DEEP * GROUPS) {
    float x[DEEP];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      const int at = b + i * GROUPS;
      x[i] = at < blocks && c < D ? part[(int64_t)at * D + c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < DEEP; ++i) s += x[i];
  }
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if ((threadIdx.x & 63) < kJoinCols) sums[threadIdx.x >> 6][l] = s;
  __syncthreads();
  if (threadIdx.x >= kJoinCols || c >= D) return;
  s = sums[0][l];
  for (int i = 1; i < kJoinWaves; ++i) s += sums[i][l];
  dw[c] = s;
}

// How a row of D elements lies: lanes a row (0: the whole block) and runs a lane.  A wave takes rows
// of up to four runs a lane (16384 x 2048 bf16 forward 22.5 us, by whole blocks 27.1; backward 34.9 and
// 37.9; 16384 x 1024 fp32 21.9 and 21.0, 30.0 and 28.9).
struct Shape {
  int G, P;
};
Shape shape_of(int D, int dtype) {
  const int E = dtype == kEltF32 ? 4 : 8;
  int G = 1;
  while (G < 64 && G * E < D) G <<= 1;
  const int P = (D + G * E - 1) / (G * E);
  if (P <= 4) return {G, P <= 2 ? P : 4};
  const int Q = (D + kThreads * E - 1) / (kThreads * E);       // 2 .. 8 for widths to 8192
  return {0, Q <= 2 ? 2 : Q <= 4 ? 4 : 8};
}

// Blocks that stay: as many as run at once, or the rows there are.
int64_t blocks_of(int64_t n, int G, int64_t most) {
  const int64_t per = G ? kThreads / G : 1, all = (n + per - 1) / per;
  return all < most ? all : most;
}
constexpr int64_t kFwdBlocks = 2048, kBwdBlocks = 1024;

template <int TY, typename F>
hipError_t by_shape(Shape s, F f) {
  using std::integral_constant;
  if (s.G) {
    if (s.P == 1) return f(integral_constant<int, 1>{}, std::false_type{});
    if (s.P == 2) return f(integral_constant<int, 2>{}, std::false_type{});
    return f(integral_constant<int, 4>{}, std::false_type{});
  }
  if (s.P == 2) return f(integral_constant<int, 2>{}, std::true_type{});
  if constexpr (TY == kEltF32)
    if (s.P == 8) return f(integral_constant<int, 8>{}, std::true_type{});
  return f(integral_constant<int, 4>{}, std::true_type{});
}

template <int MODE>
hipError_t forward(norm::Args a, int dtype, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const Shape sh = shape_of(a.D, dtype);
  a.G = sh.G;
  const unsigned blocks = (unsigned)blocks_of(a.n, sh.G, kFwdBlocks);
  return for_type(dtype, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    return by_shape<TY>(sh, [&](auto p, auto block) {
      fwd_kernel<TY, decltype(p)::value, decltype(block)::value, MODE>
          <<<blocks, kThreads, 0, s>>>(a);
      return hipGetLastError();
    });
  });
}

}  // namespace norm

hipError_t launch_rms_norm_fwd(const void* X, int dtype, int64_t xs, int64_t n, int D,
                               const void* R, int64_t rs, const float* w, float eps, void* S,
                               int64_t ss, void* Y, bool y8, int64_t ys, float* y_scale,
                               float* rstd, hipStream_t s) {
  norm::Args a{};
  a.X = X; a.xs = xs; a.R = R; a.rs = rs; a.w = w; a.n = n; a.D = D; a.eps = eps;
  a.S = S; a.ss = ss; a.Y = Y; a.ys = ys; a.y_scale = y_scale; a.rstd = rstd;
  return y8 ? norm::forward<norm::kNorm8>(a, dtype, s) : norm::forward<norm::kPlain>(a, dtype, s);
}

hipError_t launch_quantize_rows(const void* X, int dtype, int64_t xs, int64_t n, int D, void* Y,
                                int64_t ys, float* y_scale, hipStream_t s) {
  norm::Args a{};
  a.X = X; a.xs = xs; a.n = n; a.D = D; a.Y = Y; a.ys = ys; a.y_scale = y_scale;
  return norm::forward<norm::kRows8>(a, dtype, s);
}

size_t rms_norm_bwd_workspace_bytes(int64_t n, int D, int dtype) {
  const norm::Shape sh = norm::shape_of(D, dtype);
  return (size_t)norm::blocks_of(n, sh.G, norm::kBwdBlocks) * (size_t)D * 4 + 256;
}

hipError_t launch_rms_norm_bwd(const void* dY, int dtype, int64_t dys, int64_t n, int D,
                               const void* S, int64_t ss, const float* rstd, const float* w,
                               const void* dS, int64_t dss, void* dX, int64_t dxs, float* dw,
                               void* workspace, hipStream_t s) {
  norm::Args a{};
  a.dY = dY; a.dys = dys; a.n = n; a.D = D; a.X = S; a.xs = ss;
  a.rstd = const_cast<float*>(rstd); a.w = w; a.dS = dS; a.dss = dss; a.dX = dX; a.dxs = dxs;
  a.part = dw ? static_cast<float*>(workspace) : nullptr;
  const norm::Shape sh = norm::shape_of(D, dtype);
  a.G = sh.G;
  const int blocks = (int)norm::blocks_of(n, sh.G, norm::kBwdBlocks);
  if (blocks > 0) {
    const hipError_t e = for_type(dtype, [&](auto ty) {
      constexpr int TY = decltype(ty)::value;
      return norm::by_shape<TY>(sh, [&](auto p, auto block) {
        norm::bwd_kernel<TY, decltype(p)::value, decltype(block)::value>
            <<<(unsigned)blocks, norm::kThreads, 0, s>>>(a);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  if (dw)
    norm::join_kernel<<<(unsigned)((D + norm::kJoinCols - 1) / norm::kJoinCols),
                        norm::kJoinThreads, 0, s>>>(a.part, blocks, D, dw);
  return hipGetLastError();
}

}  // namespace ctr

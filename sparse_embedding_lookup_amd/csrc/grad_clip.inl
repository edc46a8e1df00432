// grad_clip.inl -- the norm of many gradients together and what is done with the clipped
// gradients.  Part of the translation unit of dense.hip.
//
//   norm = sqrt(sum over all elements g^2),  scale = norm > max_norm ? max_norm / norm : 1
//   clip: out = scale * g;   SGD step: p = p - (lr * scale) * g, rounded once at the store.
// Squares and sums are binary64: no finite binary32 gradient overflows or vanishes in its
// square.  The gradients are cut into chunks of kChunk elements that the blocks of one grid
// take in turn; each block leaves one partial sum, and each block of the second kernel adds
// all partial sums in the same order, so the norm is the same in every run and nothing waits
// on the host.  Both kernels are bound by the bytes they move (half a gigabyte of bf16 gradients
// 309 us, 5.1 TB/s over the two readings and the writing).  The second kernel takes the
// chunks last to first: those read last are the ones the 256 MB memory-side cache still holds.
namespace ctr {
namespace clip {

constexpr int kThreads = 256;
constexpr int kUnit = 8;                         // elements a thread takes at a time
constexpr int kChunk = 4096;                     // elements: two units a thread
constexpr int kTensors = 100;                    // of one launch: their records are arguments
constexpr int kMaxBlocks = 2048;                 // eight blocks a compute unit

// A tensor's chunks are counted from `shift` elements before its first, so that every unit of
// `out` but the first and the last is aligned, whatever the tensor's own alignment: gradients
// are often views of one buffer, where one odd size moves all that follow off their alignment.
// (Half a gigabyte of bf16 gradients in such a buffer, written element by element: 906 us.)
struct Tensor {
  const void* g;
  void* out;
  int64_t n;
  int32_t first;                                 // the tensor's first chunk
  int8_t gty, oty, shift, pad;
};
struct Batch {
  Tensor t[kTensors];
  int32_t num, chunks;
};
static_assert(sizeof(Batch) <= 3500, "a launch's arguments");

__device__ __forceinline__ int find_tensor(const Batch& b, int c) {
  int lo = 0, hi = b.num;                        // the last tensor whose first chunk is <= c
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.t[mid].first <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) red[w] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < kThreads / 64; ++i) v += red[i];
  __syncthreads();
  return v;
}

// Eight elements as stored.  The 16-byte accesses need the element's alignment only (the
// memory pipeline takes any), aligned ones are the fast ones.
template <int TY>
struct Unit {
  static constexpr int kElem = TY == kEltF32 ? 4 : 2, kWords = kUnit * kElem / 4;
  uint32_t u[kWords];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    __builtin_memcpy(u, static_cast<const char*>(p) + i * kElem, sizeof(u));
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    __builtin_memcpy(static_cast<char*>(p) + i * kElem, u, sizeof(u));
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (TY == kEltF32) return __uint_as_float(u[e]);
    else return e & 1 ? half_hi<TY>(u[e >> 1]) : half_lo<TY>(u[e >> 1]);
  }
  __device__ __forceinline__ void set(int e, float a, float b) {       // elements e and e + 1
    if constexpr (TY == kEltF32) {
      u[e] = __float_as_uint(a);
      u[e + 1] = __float_as_uint(b);
    } else {
      u[e >> 1] = to_half<TY, false>(a, 0u) | (to_half<TY, false>(b, 0u) << 16);
    }
  }
};

// Calls whole(r, i) for the chunk's units r of this thread that lie inside [0, n), i their
// first element, and one(i) for the single elements of those that lie partly inside.
constexpr int kUnits = kChunk / (kThreads * kUnit);
template <typename Whole, typename One>
__device__ __forceinline__ void walk(int64_t i0, int64_t n, Whole whole, One one) {
#pragma unroll
  for (int r = 0; r < kUnits; ++r) {
    const int64_t i = i0 + (r * kThreads + (int)threadIdx.x) * kUnit;
    if (i >= 0 && i + kUnit <= n) whole(r, i);
    else
      for (int e = 0; e < kUnit; ++e)
        if (i + e >= 0 && i + e < n) one(i + e);
  }
}

// The sum of squares of one chunk's elements that are this thread's.
template <int TY>
__device__ __forceinline__ double square_sum(const void* g, int64_t i0, int64_t n) {
  double s = 0.0;
  Unit<TY> x[kUnits];
  auto add = [&](double v) { s = __builtin_fma(v, v, s); };
  if (i0 >= 0 && i0 + kChunk <= n) {
#pragma unroll
    for (int r = 0; r < kUnits; ++r) x[r].load(g, i0 + (r * kThreads + (int)threadIdx.x) * kUnit);
#pragma unroll
    for (int r = 0; r < kUnits; ++r)
#pragma unroll
      for (int e = 0; e < kUnit; ++e) add(x[r].get(e));
  } else {
    walk(i0, n,
         [&](int r, int64_t i) {
           x[r].load(g, i);
#pragma unroll
           for (int e = 0; e < kUnit; ++e) add(x[r].get(e));
         },
         [&](int64_t i) { add(rows::load1<TY>(g, i)); });
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(Batch b, double* __restrict__ partial) {
  __shared__ double red[kThreads / 64];
  double s = 0.0;
  for (int c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const int i = find_tensor(b, c);
    const void* g = b.t[i].g;
    const int64_t n = b.t[i].n, i0 = (int64_t)(c - b.t[i].first) * kChunk - b.t[i].shift;
    const int ty = b.t[i].gty;
    if (ty == kEltF32) s += square_sum<kEltF32>(g, i0, n);
    else if (ty == kEltBF16) s += square_sum<kEltBF16>(g, i0, n);
    else s += square_sum<kEltF16>(g, i0, n);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// One chunk of p = f(g, p); GT and PT are the types of g and p, OLD: p is read.
template <int GT, int PT, bool OLD, typename F>
__device__ __forceinline__ void update_chunk(const void* g, void* p, int64_t i0, int64_t n, F f) {
  Unit<GT> x[kUnits];
  Unit<PT> y[kUnits];
  auto put = [&](int r, int64_t i) {
#pragma unroll
    for (int e = 0; e < kUnit; e += 2)
      y[r].set(e, f(x[r].get(e), OLD ? y[r].get(e) : 0.f),
               f(x[r].get(e + 1), OLD ? y[r].get(e + 1) : 0.f));
    y[r].store(p, i);
  };
  if (i0 >= 0 && i0 + kChunk <= n) {
#pragma unroll
    for (int r = 0; r < kUnits; ++r) {
      const int64_t i = i0 + (r * kThreads + (int)threadIdx.x) * kUnit;
      x[r].load(g, i);
      if constexpr (OLD) y[r].load(p, i);
    }
#pragma unroll
    for (int r = 0; r < kUnits; ++r)
      put(r, i0 + (r * kThreads + (int)threadIdx.x) * kUnit);
  } else {
    walk(i0, n,
         [&](int r, int64_t i) {
           x[r].load(g, i);
           if constexpr (OLD) y[r].load(p, i);
           put(r, i);
         },
         [&](int64_t i) {
           const float old = OLD ? rows::load1<PT>(p, i) : 0.f;
           rows::store1<PT>(p, i, f(rows::load1<GT>(g, i), old));
         });
  }
}

template <int GT>
__device__ __forceinline__ void sgd_by_param(int pt, const void* g, void* p, int64_t i0,
                                             int64_t n, float c) {
  auto step = [c](float x, float old) { return __builtin_fmaf(-c, x, old); };
  if (pt == kEltF32) update_chunk<GT, kEltF32, true>(g, p, i0, n, step);
  else if (pt == kEltBF16) update_chunk<GT, kEltBF16, true>(g, p, i0, n, step);
  else update_chunk<GT, kEltF16, true>(g, p, i0, n, step);
}

template <bool SGD>
__global__ __launch_bounds__(kThreads) void apply_kernel(Batch b,
                                                         const double* __restrict__ partial,
                                                         int partials, float max_norm, float lr,
                                                         float* __restrict__ stats) {
  __shared__ double red[kThreads / 64];
  double s = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
  const double norm = sqrt(block_sum(s, red));
  const double scale = norm > (double)max_norm ? (double)max_norm / norm
                                               : (norm == norm ? 1.0 : norm);
  if (stats && blockIdx.x == 0 && threadIdx.x == 0) {
    stats[0] = (float)norm;
    stats[1] = (float)scale;
  }
  const float c = (float)(SGD ? (double)lr * scale : scale);
  for (int q = b.chunks - 1 - (int)blockIdx.x; q >= 0; q -= gridDim.x) {
    const int i = find_tensor(b, q);
    const void* g = b.t[i].g;
    void* out = b.t[i].out;
    const int64_t n = b.t[i].n, i0 = (int64_t)(q - b.t[i].first) * kChunk - b.t[i].shift;
    const int gty = b.t[i].gty;
    if constexpr (SGD) {
      const int oty = b.t[i].oty;
      if (gty == kEltF32) sgd_by_param<kEltF32>(oty, g, out, i0, n, c);
      else if (gty == kEltBF16) sgd_by_param<kEltBF16>(oty, g, out, i0, n, c);
      else sgd_by_param<kEltF16>(oty, g, out, i0, n, c);
    } else {
      if (g == out && c == 1.f) continue;        // in place and not clipped: nothing to write
      auto scaled = [c](float x, float) { return x * c; };
      if (gty == kEltF32) update_chunk<kEltF32, kEltF32, false>(g, out, i0, n, scaled);
      else if (gty == kEltBF16) update_chunk<kEltBF16, kEltBF16, false>(g, out, i0, n, scaled);
      else update_chunk<kEltF16, kEltF16, false>(g, out, i0, n, scaled);
    }
  }
}

}  // namespace clip

static int64_t clip_launches(int num) { return (num + clip::kTensors - 1) / clip::kTensors; }

size_t grad_clip_workspace_bytes(int num) {
  return (size_t)(num > 0 ? clip_launches(num) : 1) * clip::kMaxBlocks * sizeof(double);
}

hipError_t launch_grad_clip(int num, const void* const* grads, const int64_t* sizes,
                            const int32_t* gtypes, void* const* outs, const int32_t* otypes,
                            bool sgd, float lr, float max_norm, float* stats, void* workspace,
                            hipStream_t s) {
  double* partial = static_cast<double*>(workspace);
  const int64_t launches = num > 0 ? clip_launches(num) : 1;
  // every block of the second pass adds up all partial sums: fewer blocks a launch where there
  // are several launches (their number enters squared: 100 tensors of 20000 fp32 elements take
  // 12 us, 500 69, 1000 145, 5000 1193)
  const int most = launches > 1 ? clip::kMaxBlocks / 2 : clip::kMaxBlocks;
  int partials = 0;
  for (int pass = 0; pass < 2; ++pass)
    // the second pass takes the launches last to first, like their chunks
    for (int64_t l = 0; l < launches; ++l) {
      const int64_t at = pass ? launches - 1 - l : l;
      clip::Batch b{};
      for (int64_t i = at * clip::kTensors; i < num && b.num < clip::kTensors; ++i) {
        if (sizes[i] == 0) continue;
        clip::Tensor& t = b.t[b.num++];
        t.g = grads[i];
        t.out = outs && outs[i] ? outs[i] : const_cast<void*>(grads[i]);
        t.n = sizes[i];
        t.first = b.chunks;
        t.gty = (int8_t)gtypes[i];
        t.oty = (int8_t)(otypes ? otypes[i] : gtypes[i]);
        const int elem = t.oty == kEltF32 ? 4 : 2;
        t.shift = (int8_t)((reinterpret_cast<uintptr_t>(t.out) & 15u) / elem);
        b.chunks += (int32_t)((sizes[i] + t.shift + clip::kChunk - 1) / clip::kChunk);
      }
      const int blocks = b.chunks < most ? b.chunks : most;
      if (pass == 0) {
        if (blocks == 0) continue;
        clip::norm_kernel<<<blocks, clip::kThreads, 0, s>>>(b, partial + partials);
        partials += blocks;
      } else {
        float* st = l == 0 ? stats : nullptr;
        if (blocks == 0 && !st) continue;
        const int grid = blocks > 0 ? blocks : 1;
        if (sgd)
          clip::apply_kernel<true><<<grid, clip::kThreads, 0, s>>>(b, partial, partials, max_norm,
                                                                   lr, st);
        else
          clip::apply_kernel<false><<<grid, clip::kThreads, 0, s>>>(b, partial, partials,
                                                                    max_norm, lr, st);
      }
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace ctr

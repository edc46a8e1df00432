// grad_clip.inl -- the norm of many gradients together and what is done with the clipped
// gradients.  Part of the translation unit of dense.hip.
//
//   norm = sqrt(sum over all elements g^2),  scale = norm > max_norm ? max_norm / norm : 1
//   clip: out = scale * g;   SGD step: p = p - (lr * scale) * g, rounded once at the store.
// Squares and sums are binary64: no finite binary32 gradient overflows or vanishes in its
// square.  The gradients are cut into chunks of kChunk elements that the blocks of one grid
// take in turn; each block leaves one partial sum, and each block of the second kernel adds
// all partial sums in the same order, so the norm is the same in every run and nothing waits
// on the host.  Both kernels are bound by the bytes they move.  The second kernel takes the
// chunks last to first: those read last are the ones the 256 MB memory-side cache still holds.
namespace ctr {
namespace clip {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;                     // elements: 32 a thread
constexpr int kTensors = 100;                    // of one launch: their records are arguments
constexpr int kMaxBlocks = 1024;                 // four blocks a compute unit

struct Tensor {
  const void* g;
  void* out;
  int64_t n;
  int32_t first;                                 // the tensor's first chunk
  int8_t gty, oty, vec, pad;
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

// The sum of squares of one chunk's elements that are this thread's.
template <int TY>
__device__ __forceinline__ double square_sum(const void* g, int64_t i0, int64_t n, bool vec) {
  double s = 0.0;
  const int64_t end = n < i0 + kChunk ? n : i0 + kChunk;
  if (vec && end - i0 == kChunk) {
    constexpr int W = Vec<TY>::kElems, R = kChunk / (kThreads * W);
    Vec<TY> x[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      x[r].load(static_cast<const char*>(g) +
                (i0 + (int64_t)(r * kThreads + threadIdx.x) * W) * (TY == kEltF32 ? 4 : 2));
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < W; ++e) s = __builtin_fma((double)x[r].v[e], (double)x[r].v[e], s);
  } else {
    for (int64_t i = i0 + threadIdx.x; i < end; i += kThreads) {
      const double v = rows::load1<TY>(g, i);
      s = __builtin_fma(v, v, s);
    }
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(Batch b, double* __restrict__ partial) {
  __shared__ double red[kThreads / 64];
  double s = 0.0;
  for (int c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const int i = find_tensor(b, c);
    const void* g = b.t[i].g;
    const int64_t n = b.t[i].n, i0 = (int64_t)(c - b.t[i].first) * kChunk;
    const bool vec = b.t[i].vec;
    const int ty = b.t[i].gty;
    if (ty == kEltF32) s += square_sum<kEltF32>(g, i0, n, vec);
    else if (ty == kEltBF16) s += square_sum<kEltBF16>(g, i0, n, vec);
    else s += square_sum<kEltF16>(g, i0, n, vec);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

template <int TY>
__device__ __forceinline__ void scale_chunk(const void* g, void* out, int64_t i0, int64_t n,
                                            bool vec, float c) {
  const int64_t end = n < i0 + kChunk ? n : i0 + kChunk;
  if (vec && end - i0 == kChunk) {
    using P = rows::Piece<TY, true>;
    constexpr int W = P::kElems, R = kChunk / (kThreads * W);
    P x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r].load(g, i0 + (int64_t)(r * kThreads + threadIdx.x) * W);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < W; ++e) x[r].v[e] *= c;
      x[r].store(out, i0 + (int64_t)(r * kThreads + threadIdx.x) * W);
    }
  } else {
    for (int64_t i = i0 + threadIdx.x; i < end; i += kThreads)
      rows::store1<TY>(out, i, rows::load1<TY>(g, i) * c);
  }
}

template <int GT, int PT>
__device__ __forceinline__ void sgd_chunk(const void* g, void* p, int64_t i0, int64_t n, bool vec,
                                          float c) {
  const int64_t end = n < i0 + kChunk ? n : i0 + kChunk;
  if (vec && end - i0 == kChunk) {
    // eight elements a thread and round, whatever the types
    constexpr int R = kChunk / (kThreads * 8);
    using G = rows::Piece<GT, true>;
    using P = rows::Piece<PT, true>;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t i = i0 + (int64_t)(r * kThreads + threadIdx.x) * 8;
      float x[8];
#pragma unroll
      for (int q = 0; q < 8 / G::kElems; ++q) {
        G v;
        v.load(g, i + q * G::kElems);
#pragma unroll
        for (int e = 0; e < G::kElems; ++e) x[q * G::kElems + e] = v.v[e];
      }
#pragma unroll
      for (int q = 0; q < 8 / P::kElems; ++q) {
        P v;
        v.load(p, i + q * P::kElems);
#pragma unroll
        for (int e = 0; e < P::kElems; ++e)
          v.v[e] = __builtin_fmaf(-c, x[q * P::kElems + e], v.v[e]);
        v.store(p, i + q * P::kElems);
      }
    }
  } else {
    for (int64_t i = i0 + threadIdx.x; i < end; i += kThreads)
      rows::store1<PT>(p, i, __builtin_fmaf(-c, rows::load1<GT>(g, i), rows::load1<PT>(p, i)));
  }
}

template <int GT>
__device__ __forceinline__ void sgd_by_param(int pt, const void* g, void* p, int64_t i0,
                                             int64_t n, bool vec, float c) {
  if (pt == kEltF32) sgd_chunk<GT, kEltF32>(g, p, i0, n, vec, c);
  else if (pt == kEltBF16) sgd_chunk<GT, kEltBF16>(g, p, i0, n, vec, c);
  else sgd_chunk<GT, kEltF16>(g, p, i0, n, vec, c);
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
    const int64_t n = b.t[i].n, i0 = (int64_t)(q - b.t[i].first) * kChunk;
    const bool vec = b.t[i].vec;
    const int gty = b.t[i].gty;
    if constexpr (SGD) {
      const int oty = b.t[i].oty;
      if (gty == kEltF32) sgd_by_param<kEltF32>(oty, g, out, i0, n, vec, c);
      else if (gty == kEltBF16) sgd_by_param<kEltBF16>(oty, g, out, i0, n, vec, c);
      else sgd_by_param<kEltF16>(oty, g, out, i0, n, vec, c);
    } else {
      if (g == out && c == 1.f) continue;        // in place and not clipped: nothing to write
      if (gty == kEltF32) scale_chunk<kEltF32>(g, out, i0, n, vec, c);
      else if (gty == kEltBF16) scale_chunk<kEltBF16>(g, out, i0, n, vec, c);
      else scale_chunk<kEltF16>(g, out, i0, n, vec, c);
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
        t.vec = ((reinterpret_cast<uintptr_t>(t.g) | reinterpret_cast<uintptr_t>(t.out)) & 15u) == 0;
        b.chunks += (int32_t)((sizes[i] + clip::kChunk - 1) / clip::kChunk);
      }
      const int blocks = b.chunks < clip::kMaxBlocks ? b.chunks : clip::kMaxBlocks;
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

// expert_rows.inl -- rows on their way to the experts and back: the router, the sort of the
// slots by expert, the copy of rows into that order, the weighted sum back, and the gradients
// of all of them.  Part of the translation unit of dense.hip.
//
// A token t has k slots (t, j), flat index i = t*k + j; slot i goes to expert experts[i], or
// nowhere when that is not in [0, E) (a dropped slot).  The sorted order lists the slots by
// expert, those of one expert in slot order; position p holds slot order[p], and slots[i] is
// the position of slot i (-1 dropped).  offsets[e] is expert e's first position, offsets[E]
// the number of slots that have one; order is -1 from there on.
namespace ctr {
namespace rows {

constexpr int kThreads = 256;

// ------------------------------------------------------------------------------- router
// G lanes (a power of two, at least k and at most 64) hold one row of E logits, V a lane:
// lane l holds experts V l .. V l + V - 1, which it reads and writes together.  The k largest
// are taken one at a time: each lane's best of what it has left, joined over the lanes by a
// butterfly that prefers the larger value and, among equals, the lower expert; lane j keeps the
// j-th.  The softmax is relative to the first value taken, the row's largest.  A logit that is
// -inf or NaN closes its expert.
// Bound by the instructions of the k rounds: forward 8.6 us, backward, whose k entries of a token
// are exchanged through LDS, 6.1 us at 65536 x 64 bf16, 4 experts (bytes: 2 us each).  A wave has
// 440 and 206 vector instructions, eight waves a SIMD: 5.9 and 2.7 us of issue at 2.4 GHz.  With
// the forward's exchanges through LDS and one logit a load 10.7 and 7.1 us.
template <int TY>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (TY == kEltF32) return static_cast<const float*>(p)[i];
  else return half_lo<TY>(static_cast<const uint16_t*>(p)[i]);
}
template <int TY>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (TY == kEltF32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)to_half<TY, false>(v, 0u);
}

__device__ __forceinline__ float ninf() { return __uint_as_float(0xFF800000u); }

// exp(x - m) for x <= m, also where both are infinite
__device__ __forceinline__ float exp_below(float x, float m) {
  return x == m ? 1.f : expf(x - m);
}

// Calls f(get) for every step of a butterfly over G lanes, get(v) the other lane's v: within 16
// lanes by the data-parallel moves (the mirrors of 8 and 16 lanes do as steps of 4 and 8 where
// all lanes of a group already hold the same), which take no trip through LDS.
template <int CTRL>
__device__ __forceinline__ int moved(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}
template <typename F>
__device__ __forceinline__ void butterfly(int G, F f) {
  if (G > 1) f([](int v) { return moved<0xB1>(v); });          // quads 1 0 3 2
  if (G > 2) f([](int v) { return moved<0x4E>(v); });          // quads 2 3 0 1
  if (G > 4) f([](int v) { return moved<0x141>(v); });         // half rows mirrored
  if (G > 8) f([](int v) { return moved<0x140>(v); });         // rows mirrored
  if (G > 16) f([](int v) { return __shfl_xor(v, 16); });
  if (G > 32) f([](int v) { return __shfl_xor(v, 32); });
}
__device__ __forceinline__ float group_sum(int G, float v) {
  butterfly(G, [&](auto get) { v += __int_as_float(get(__float_as_int(v))); });
  return v;
}

// A lane's V logits, those from n on as `none`; V of them at a row's place `first`.
template <int TY, int V>
__device__ __forceinline__ void load_lane(const void* row, int first, int n, float none, float* x) {
  constexpr int SIZE = TY == kEltF32 ? 4 : 2;
  if constexpr (V * SIZE >= 4) {
    if (first + V <= n) {
      uint32_t u[V * SIZE / 4];
      __builtin_memcpy(u, static_cast<const char*>(row) + (int64_t)first * SIZE, sizeof(u));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (TY == kEltF32) x[i] = __uint_as_float(u[i]);
        else x[i] = i & 1 ? half_hi<TY>(u[i >> 1]) : half_lo<TY>(u[i >> 1]);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = first + i < n ? load1<TY>(row, first + i) : none;
}
template <int TY, int V>
__device__ __forceinline__ void store_lane(void* row, int first, int n, const float* x) {
  constexpr int SIZE = TY == kEltF32 ? 4 : 2;
  if constexpr (V * SIZE >= 4) {
    if (first + V <= n) {
      uint32_t u[V * SIZE / 4];
#pragma unroll
      for (int i = 0; i < V * SIZE / 4; ++i) {
        if constexpr (TY == kEltF32) u[i] = __float_as_uint(x[i]);
        else u[i] = to_half<TY, false>(x[2 * i], 0u) | (to_half<TY, false>(x[2 * i + 1], 0u) << 16);
      }
      __builtin_memcpy(static_cast<char*>(row) + (int64_t)first * SIZE, u, sizeof(u));
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (first + i < n) store1<TY>(row, first + i, x[i]);
}
// Row t of a matrix of element type TY and row stride s.
template <int TY>
__device__ __forceinline__ const void* row_of(const void* p, int64_t t, int64_t s) {
  return static_cast<const char*>(p) + t * s * (TY == kEltF32 ? 4 : 2);
}

template <int TY, int V>
__global__ __launch_bounds__(kThreads) void route_fwd_kernel(
    const void* __restrict__ logits, int64_t ls, int64_t T, int E, int k, int G, int renorm,
    int32_t* __restrict__ experts, float* __restrict__ weights) {
  const int l = threadIdx.x & (G - 1);
  const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / G;
  const bool row = t < T;
  float x[V];
  load_lane<TY, V>(row_of<TY>(logits, t, ls), l * V, row ? E : 0, ninf(), x);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = x[i] > ninf() ? x[i] : ninf();      // NaN too
  float most = 0.f, total = 0.f, mine = ninf();
  int chosen = -1;
  for (int j = 0; j < k; ++j) {
    float best = ninf();
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (x[i] > best) {
        best = x[i];
        at = l * V + i;
      }
    butterfly(G, [&](auto get) {
      const float v = __int_as_float(get(__float_as_int(best)));
      const int a = get(at);
      if (v > best || (v == best && a < at)) {
        best = v;
        at = a;
      }
    });
    if (j == 0) {
      most = best;
      if (!renorm) {
#pragma unroll
        for (int i = 0; i < V; ++i) total += x[i] > ninf() ? exp_below(x[i], most) : 0.f;
        total = group_sum(G, total);
      }
    }
    if (renorm && best > ninf()) total += exp_below(best, most);
    if (l == j && best > ninf()) {
      mine = best;
      chosen = at;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (l * V + i == at) x[i] = ninf();
  }
  if (row && l < k) {
    experts[t * k + l] = chosen;
    weights[t * k + l] = chosen >= 0 ? exp_below(mine, most) / total : 0.f;
  }
}

// With q the softmax the weights were taken from (over the chosen experts when renorm, over
// all else) and s = sum_j w_j dw_j: dlogit_e = q_e (dw of e if chosen, else 0, minus s).
template <int TY, int V>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(
    const void* __restrict__ logits, int64_t ls, int64_t T, int E, int k, int G, int renorm,
    const int32_t* __restrict__ experts, const float* __restrict__ weights,
    const float* __restrict__ dweights, void* __restrict__ dlogits, int64_t dls) {
  const int l = threadIdx.x & (G - 1);
  const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / G;
  const bool row = t < T;
  int chosen = -1;
  float w = 0.f, dw = 0.f;
  if (row && l < k) {
    chosen = experts[t * k + l];
    if (chosen >= 0 && chosen < E) {
      w = weights[t * k + l];
      dw = dweights[t * k + l];
    } else {
      chosen = -1;
    }
  }
  const float s = group_sum(G, w * dw);
  float q[V], g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) q[i] = g[i] = 0.f;
  if (!renorm) {
    float most = ninf(), total = 0.f;
    load_lane<TY, V>(row_of<TY>(logits, t, ls), l * V, row ? E : 0, ninf(), q);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      q[i] = q[i] > ninf() ? q[i] : ninf();
      most = fmaxf(most, q[i]);
    }
    butterfly(G, [&](auto get) { most = fmaxf(most, __int_as_float(get(__float_as_int(most)))); });
#pragma unroll
    for (int i = 0; i < V; ++i) {
      q[i] = q[i] > ninf() ? exp_below(q[i], most) : 0.f;
      total += q[i];
    }
    total = group_sum(G, total);
    const float by = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] *= by;
  }
  const int first = (threadIdx.x & 63) & ~(G - 1);
  for (int j = 0; j < k; ++j) {
    const int e = __shfl(chosen, first + j);
    const float wj = __shfl(w, first + j), dj = __shfl(dw, first + j);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (l * V + i == e) {
        g[i] = dj;
        if (renorm) q[i] = wj;
      }
  }
  if (!row) return;
#pragma unroll
  for (int i = 0; i < V; ++i) q[i] *= g[i] - s;
  store_lane<TY, V>(const_cast<void*>(row_of<TY>(dlogits, t, dls)), l * V, E, q);
}

// --------------------------------------------------------------------------------- sort
// A counting sort in two launches, or one when a block holds every slot.  Block b has the
// slots [b*chunk, (b+1)*chunk), its wave w a contiguous part of them.  The first launch counts
// the block's slots of each expert.  In the second every block adds up the counts of the
// blocks before it and of the experts before each expert, its waves count their own slots,
// and each wave then walks its slots 64 at a time: a lane's place among the lanes of the same
// expert comes from a ballot per key bit, so the order within an expert is the slots' own.
// Bound by the launches and the steps of a block, not by its 12 bytes a slot: 2.7 and 4.9 us for
// 16384 slots, 4.8 and 10.8 us for 65542 (one launch, 74 slots: 3.2 us).  Many experts make the
// walk over all blocks' counts, blocks x E cells with two divisions each in every block, the
// larger part: 131072 slots take 18.7 us with 64 experts and 196 us with 1024 (both launches).
constexpr int kSortThreads = 512, kSortWaves = kSortThreads / kWave;

__device__ __forceinline__ int sort_key(const int32_t* experts, int64_t i, int64_t end, int E) {
  const int e = i < end ? experts[i] : -1;
  return e >= 0 && e < E ? e : E;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(
    const int32_t* __restrict__ experts, int64_t n, int E, int64_t chunk,
    int32_t* __restrict__ counts) {
  extern __shared__ int32_t hist[];
  for (int e = threadIdx.x; e <= E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * chunk, end = n < begin + chunk ? n : begin + chunk;
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads)
    atomicAdd(&hist[sort_key(experts, i, end, E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(
    const int32_t* __restrict__ experts, int64_t n, int E, int bits, int64_t chunk,
    const int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
    int32_t* __restrict__ slots, int32_t* __restrict__ order) {
  // next[w][e]: wave w's next position for expert e; all[e], before[e]: slots of expert e in
  // all blocks, and in the blocks before this one
  extern __shared__ int32_t lds[];
  int32_t* next = lds;
  int32_t* all = lds + kSortWaves * (E + 1);
  int32_t* before = all + E + 1;
  __shared__ int32_t carry[kSortWaves + 1];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t begin = blockIdx.x * chunk;
  const int64_t part = chunk / kSortWaves;
  const int64_t wb = begin + w * part;
  int64_t we = wb + part;
  if (we > n) we = n;
  for (int i = tid; i < kSortWaves * (E + 1); i += kSortThreads) next[i] = 0;
  for (int e = tid; e <= E; e += kSortThreads) all[e] = before[e] = 0;
  __syncthreads();
  for (int64_t i = wb + lane; i < we; i += kWave)
    atomicAdd(&next[w * (E + 1) + sort_key(experts, i, we, E)], 1);
  __syncthreads();
  if (gridDim.x == 1) {
    for (int e = tid; e < E; e += kSortThreads) {
      int32_t s = 0;
      for (int v = 0; v < kSortWaves; ++v) s += next[v * (E + 1) + e];
      all[e] = s;
    }
  } else {
    // the block walks the cells of all blocks' counts, one a thread at a time
    const int64_t cells = (int64_t)gridDim.x * E;
    for (int64_t c = tid; c < cells; c += kSortThreads) {
      const int32_t v = counts[c];
      const int e = (int)(c % E);
      if (v) {
        atomicAdd(&all[e], v);
        if (c / E < blockIdx.x) atomicAdd(&before[e], v);
      }
    }
  }
  __syncthreads();
  // exclusive prefix of all over the experts, kSortThreads at a time
  int32_t run = 0;
  for (int e0 = 0; e0 < E; e0 += kSortThreads) {
    const int e = e0 + tid;
    const int32_t mine = e < E ? all[e] : 0;
    int32_t s = mine;
    for (int d = 1; d < kWave; d <<= 1) {
      const int32_t v = __shfl_up(s, d);
      if (lane >= d) s += v;
    }
    if (lane == 63) carry[w + 1] = s;
    __syncthreads();
    int32_t base = run;
    for (int v = 0; v < w; ++v) base += carry[v + 1];
    int32_t sum = 0;
    for (int v = 0; v < kSortWaves; ++v) sum += carry[v + 1];
    run += sum;
    if (e < E) {
      const int32_t at = base + s - mine;
      if (blockIdx.x == 0) offsets[e] = at;
      int32_t p = at + before[e];
      for (int v = 0; v < kSortWaves; ++v) {
        const int32_t c = next[v * (E + 1) + e];
        next[v * (E + 1) + e] = p;
        p += c;
      }
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) offsets[E] = run;
  for (int64_t p = run + (int64_t)blockIdx.x * kSortThreads + tid; p < n;
       p += (int64_t)gridDim.x * kSortThreads)
    order[p] = -1;
  for (int64_t i0 = wb; i0 < we; i0 += kWave) {
    const int64_t i = i0 + lane;
    const int key = sort_key(experts, i, we, E);
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int32_t* slot = &next[w * (E + 1) + key];
    const int32_t base = *(volatile int32_t*)slot;
    __builtin_amdgcn_wave_barrier();
    if (rank == 0) *(volatile int32_t*)slot = base + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (i < we) {
      const int32_t p = key < E ? base + rank : -1;
      slots[i] = p;
      if (p >= 0) order[p] = (int32_t)i;
    }
  }
}

// ------------------------------------------------------------------ rows there and back
// G lanes (a power of two) have one token and walk its row in pieces of 16 bytes, U of them at
// a time, so that the loads of U pieces of K slots' rows are in flight together; the last
// elements, less than a piece, go one by one.  These kernels are copies with little arithmetic,
// bound by the memory they touch: at 32771 x 2208 fp16, two slots a token, a tenth dropped,
// dispatch 78 us, combine 94 us, its gradient with that of the weights 143 us (5.6, 4.3 and 4.9
// TB/s).  A piece needs the alignment of its elements only (the memory
// pipeline takes any), so odd widths and strides run at nearly the same rate.
template <int TY, bool VEC>
struct Piece {
  static constexpr int kElems = VEC ? Vec<TY>::kElems : 1;
  float v[kElems];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    if constexpr (!VEC) {
      v[0] = load1<TY>(base, i);
    } else {
      uint32_t u[4];
      __builtin_memcpy(u, static_cast<const char*>(base) + i * (TY == kEltF32 ? 4 : 2), 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (TY == kEltF32) {
          v[e] = __uint_as_float(u[e]);
        } else {
          v[2 * e] = half_lo<TY>(u[e]);
          v[2 * e + 1] = half_hi<TY>(u[e]);
        }
      }
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    if constexpr (!VEC) {
      store1<TY>(base, i, v[0]);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (TY == kEltF32)
          u[e] = __float_as_uint(v[e]);
        else
          u[e] = to_half<TY, false>(v[2 * e], 0u) | (to_half<TY, false>(v[2 * e + 1], 0u) << 16);
      }
      __builtin_memcpy(static_cast<char*>(base) + i * (TY == kEltF32 ? 4 : 2), u, 16);
    }
  }
};

struct RowArgs {
  int64_t T, n;                 // tokens, and positions (T * k)
  int D, k, G, E;
  const int32_t* slots;
  const int32_t* offsets;       // nullable where no tail is written
  const float* weights;         // nullable: 1
  float* dweights;              // combine_bwd, nullable
  const void* x;                // dispatch: X; combine_fwd: P; combine_bwd: dY
  int64_t xs;
  const void* p;                // combine_bwd: P (nullable without dweights)
  int64_t ps;
  void* y;                      // dispatch: P; combine_fwd: Y; combine_bwd: dP
  int64_t ys;
};

// The lane's part of a row: whole(c, pieces) for its pieces c, c + G, .. U at a time, those below
// `pieces`, then one(i) for its single elements.
template <int U, int PE, typename Whole, typename One>
__device__ __forceinline__ void walk_row(const RowArgs& a, int l, Whole whole, One one) {
  const int pieces = a.D / PE;
  for (int c = l; c < pieces; c += U * a.G) whole(c, pieces);
  for (int i = pieces * PE + l; i < a.D; i += a.G) one(i);
}

// The rows of positions that hold no slot are zero.
template <int TY>
__device__ __forceinline__ void zero_tail(const RowArgs& a, int64_t t, int l) {
  using P = Piece<TY, true>;
  int64_t p = a.offsets[a.E];
  p = (p < 0 ? 0 : p) + t;
  for (; p < a.n; p += a.T)
    walk_row<1, P::kElems>(
        a, l, [&](int c, int) { P{}.store(a.y, p * a.ys + c * P::kElems); },
        [&](int i) { store1<TY>(a.y, p * a.ys + i, 0.f); });
}

// The positions (-1: none) and weights of K of a token's slots, from slot j on.
template <int K>
struct Slots {
  int64_t p[K];
  float w[K];
  __device__ __forceinline__ void load(const RowArgs& a, int64_t t, int j) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int64_t at = j + i < a.k ? a.slots[t * a.k + j + i] : -1;
      p[i] = at >= 0 && at < a.n ? at : -1;
      w[i] = a.weights && j + i < a.k ? a.weights[t * a.k + j + i] : 1.f;
    }
  }
};

template <int TY, int K>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(RowArgs a) {
  const int l = threadIdx.x & (a.G - 1);
  const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / a.G;
  if (t >= a.T) return;
  using P = Piece<TY, true>;
  constexpr int PE = P::kElems, U = 4;
  for (int j = 0; j < a.k; j += K) {
    Slots<K> s;
    s.load(a, t, j);
    walk_row<U, PE>(
        a, l,
        [&](int c, int pieces) {
          P x[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c + u * a.G < pieces) x[u].load(a.x, t * a.xs + (c + u * a.G) * PE);
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (s.p[i] >= 0)
#pragma unroll
              for (int u = 0; u < U; ++u)
                if (c + u * a.G < pieces) x[u].store(a.y, s.p[i] * a.ys + (c + u * a.G) * PE);
        },
        [&](int e) {
          const float x = load1<TY>(a.x, t * a.xs + e);
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (s.p[i] >= 0) store1<TY>(a.y, s.p[i] * a.ys + e, x);
        });
  }
  zero_tail<TY>(a, t, l);
}

template <int TY, int K>
__global__ __launch_bounds__(kThreads) void combine_fwd_kernel(RowArgs a) {
  const int l = threadIdx.x & (a.G - 1);
  const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / a.G;
  if (t >= a.T) return;
  using P = Piece<TY, true>;
  // one piece of each of the K rows: 9.5 us at 8192 x 1024 and 94 us at 32771 x 2208, with two
  // pieces 10.4 and 92 us, with four 11.9 and 114 us (fewer waves at once)
  constexpr int PE = P::kElems, U = 1;
  Slots<K> s;
  s.load(a, t, 0);
  walk_row<U, PE>(
      a, l,
      [&](int c, int pieces) {
        P y[U]{};
        for (int j = 0; j < a.k; j += K) {
          if (a.k > K) s.load(a, t, j);
          P x[K][U];
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (s.p[i] >= 0)
#pragma unroll
              for (int u = 0; u < U; ++u)
                if (c + u * a.G < pieces) x[i][u].load(a.x, s.p[i] * a.xs + (c + u * a.G) * PE);
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (s.p[i] >= 0)
#pragma unroll
              for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < PE; ++e)
                  y[u].v[e] = __builtin_fmaf(s.w[i], x[i][u].v[e], y[u].v[e]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c + u * a.G < pieces) y[u].store(a.y, t * a.ys + (c + u * a.G) * PE);
      },
      [&](int e) {
        float y = 0.f;
        for (int j = 0; j < a.k; j += K) {
          if (a.k > K) s.load(a, t, j);
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (s.p[i] >= 0) y = __builtin_fmaf(s.w[i], load1<TY>(a.x, s.p[i] * a.xs + e), y);
        }
        store1<TY>(a.y, t * a.ys + e, y);
      });
}

template <int TY, int K>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(RowArgs a) {
  const int l = threadIdx.x & (a.G - 1);
  const int64_t t = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / a.G;
  if (t >= a.T) return;
  using P = Piece<TY, true>;
  constexpr int PE = P::kElems, U = 2;
  for (int j = 0; j < a.k; j += K) {
    Slots<K> s;
    s.load(a, t, j);
    float dot[K];
#pragma unroll
    for (int i = 0; i < K; ++i) dot[i] = 0.f;
    walk_row<U, PE>(
        a, l,
        [&](int c, int pieces) {
          P g[U], x[K][U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c + u * a.G < pieces) g[u].load(a.x, t * a.xs + (c + u * a.G) * PE);
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (s.p[i] >= 0 && a.dweights)
#pragma unroll
              for (int u = 0; u < U; ++u)
                if (c + u * a.G < pieces) x[i][u].load(a.p, s.p[i] * a.ps + (c + u * a.G) * PE);
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (s.p[i] >= 0)
#pragma unroll
              for (int u = 0; u < U; ++u)
                if (c + u * a.G < pieces) {
                  P d;
#pragma unroll
                  for (int e = 0; e < PE; ++e) {
                    if (a.dweights) dot[i] = __builtin_fmaf(g[u].v[e], x[i][u].v[e], dot[i]);
                    d.v[e] = s.w[i] * g[u].v[e];
                  }
                  d.store(a.y, s.p[i] * a.ys + (c + u * a.G) * PE);
                }
        },
        [&](int e) {
          const float g = load1<TY>(a.x, t * a.xs + e);
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (s.p[i] >= 0) {
              if (a.dweights)
                dot[i] = __builtin_fmaf(g, load1<TY>(a.p, s.p[i] * a.ps + e), dot[i]);
              store1<TY>(a.y, s.p[i] * a.ys + e, s.w[i] * g);
            }
        });
    if (a.dweights) {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        for (int d = 1; d < a.G; d <<= 1) dot[i] += __shfl_xor(dot[i], d);
        if (l == 0 && j + i < a.k) a.dweights[t * a.k + j + i] = dot[i];
      }
    }
  }
  zero_tail<TY>(a, t, l);
}

}  // namespace rows

// Logits a lane holds: up to 8, as a lane's own comparisons cost less than a step of the
// butterfly, and 16 where 64 lanes of 8 do not hold a row.
static int route_values(int E) {
  int V = E <= 8 ? 1 : E <= 16 ? 2 : E <= 32 ? 4 : 8;
  while (V * 64 < E) V *= 2;
  return V;
}
static int route_group(int E, int k, int V) {
  int G = 1;
  while (G < k || G * V < E) G <<= 1;
  return G;
}

template <typename F>
static hipError_t by_values(int V, F f) {
  switch (V) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    default: return f(std::integral_constant<int, 16>{});
  }
}
template <typename F>
static hipError_t by_type(int dtype, F f) {
  if (dtype == kEltF32) return f(std::integral_constant<int, kEltF32>{});
  if (dtype == kEltBF16) return f(std::integral_constant<int, kEltBF16>{});
  return f(std::integral_constant<int, kEltF16>{});
}

hipError_t launch_expert_route_fwd(const void* logits, int dtype, int64_t ls, int64_t T, int E,
                                   int k, bool renorm, int32_t* experts, float* weights,
                                   hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int V = route_values(E), G = route_group(E, k, V);
  const unsigned blocks = (unsigned)((T * G + rows::kThreads - 1) / rows::kThreads);
  return by_type(dtype, [&](auto ty) {
    return by_values(V, [&](auto v) {
      rows::route_fwd_kernel<decltype(ty)::value, decltype(v)::value>
          <<<blocks, rows::kThreads, 0, s>>>(logits, ls, T, E, k, G, renorm, experts, weights);
      return hipGetLastError();
    });
  });
}

hipError_t launch_expert_route_bwd(const void* logits, int dtype, int64_t ls, int64_t T, int E,
                                   int k, bool renorm, const int32_t* experts,
                                   const float* weights, const float* dweights, void* dlogits,
                                   int64_t dls, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int V = route_values(E), G = route_group(E, k, V);
  const unsigned blocks = (unsigned)((T * G + rows::kThreads - 1) / rows::kThreads);
  return by_type(dtype, [&](auto ty) {
    return by_values(V, [&](auto v) {
      rows::route_bwd_kernel<decltype(ty)::value, decltype(v)::value>
          <<<blocks, rows::kThreads, 0, s>>>(logits, ls, T, E, k, G, renorm, experts, weights,
                                             dweights, dlogits, dls);
      return hipGetLastError();
    });
  });
}

// Slots a block sorts: everything up to 4096 in one block; else at least 512 (one load a
// thread), in at most 256 blocks.
static int64_t sort_chunk(int64_t n) {
  if (n <= 4096) return n > 0 ? (n + rows::kSortThreads - 1) / rows::kSortThreads * rows::kSortThreads
                              : rows::kSortThreads;
  int64_t c = (n + 255) / 256;
  return (c + rows::kSortThreads - 1) / rows::kSortThreads * rows::kSortThreads;
}

size_t expert_sort_workspace_bytes(int64_t n, int E) {
  const int64_t c = sort_chunk(n), blocks = (n + c - 1) / c;
  return blocks > 1 ? (size_t)blocks * E * sizeof(int32_t) : 256;
}

hipError_t launch_expert_sort(const int32_t* experts, int64_t n, int E, int32_t* offsets,
                              int32_t* slots, int32_t* order, void* workspace, hipStream_t s) {
  const int64_t chunk = sort_chunk(n);
  const unsigned blocks = n > 0 ? (unsigned)((n + chunk - 1) / chunk) : 1u;
  int32_t* counts = static_cast<int32_t*>(workspace);
  if (blocks > 1) {
    rows::sort_count_kernel<<<blocks, rows::kSortThreads, (E + 1) * sizeof(int32_t), s>>>(
        experts, n, E, chunk, counts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  int bits = 1;                                    // keys 0 .. E
  while ((1 << bits) <= E) ++bits;
  const size_t lds = (size_t)(rows::kSortWaves + 2) * (E + 1) * sizeof(int32_t);
  rows::sort_place_kernel<<<blocks, rows::kSortThreads, lds, s>>>(experts, n, E, bits, chunk,
                                                                  counts, offsets, slots, order);
  return hipGetLastError();
}

// Lanes a token's row takes: as many as it has pieces, at most a wave.
static int row_lanes(int64_t pieces) {
  int G = 1;
  while (G < 64 && G < pieces) G <<= 1;
  return G;
}

template <typename F>
static hipError_t launch_rows(rows::RowArgs& a, int dtype, F f) {
  if (a.T == 0) return hipSuccess;
  a.G = row_lanes(a.D / (dtype == kEltF32 ? 4 : 8));
  const unsigned blocks = (unsigned)((a.T * a.G + rows::kThreads - 1) / rows::kThreads);
  return by_type(dtype, [&](auto ty) {
    // slots taken together: all there are up to two, else four at a time
    if (a.k == 1) f(ty, std::integral_constant<int, 1>{}, blocks);
    else if (a.k == 2) f(ty, std::integral_constant<int, 2>{}, blocks);
    else f(ty, std::integral_constant<int, 4>{}, blocks);
    return hipGetLastError();
  });
}

hipError_t launch_expert_dispatch(const void* X, int dtype, int64_t xs, int64_t T, int k, int D,
                                  const int32_t* slots, const int32_t* offsets, int E, void* P,
                                  int64_t ps, hipStream_t s) {
  rows::RowArgs a{};
  a.T = T; a.n = T * k; a.D = D; a.k = k; a.E = E;
  a.slots = slots; a.offsets = offsets;
  a.x = X; a.xs = xs; a.y = P; a.ys = ps;
  return launch_rows(a, dtype, [&](auto ty, auto k, unsigned blocks) {
    rows::dispatch_kernel<decltype(ty)::value, decltype(k)::value>
        <<<blocks, rows::kThreads, 0, s>>>(a);
  });
}

hipError_t launch_expert_combine_fwd(const void* P, int dtype, int64_t ps, int64_t T, int k,
                                     int D, const int32_t* slots, const float* weights, void* Y,
                                     int64_t ys, hipStream_t s) {
  rows::RowArgs a{};
  a.T = T; a.n = T * k; a.D = D; a.k = k;
  a.slots = slots; a.weights = weights;
  a.x = P; a.xs = ps; a.y = Y; a.ys = ys;
  return launch_rows(a, dtype, [&](auto ty, auto k, unsigned blocks) {
    rows::combine_fwd_kernel<decltype(ty)::value, decltype(k)::value>
        <<<blocks, rows::kThreads, 0, s>>>(a);
  });
}

hipError_t launch_expert_combine_bwd(const void* dY, int dtype, int64_t dys, int64_t T, int k,
                                     int D, const void* P, int64_t ps, const int32_t* slots,
                                     const int32_t* offsets, int E, const float* weights,
                                     void* dP, int64_t dps, float* dweights, hipStream_t s) {
  rows::RowArgs a{};
  a.T = T; a.n = T * k; a.D = D; a.k = k; a.E = E;
  a.slots = slots; a.offsets = offsets; a.weights = weights; a.dweights = dweights;
  a.x = dY; a.xs = dys; a.p = dweights ? P : nullptr; a.ps = ps; a.y = dP; a.ys = dps;
  return launch_rows(a, dtype, [&](auto ty, auto k, unsigned blocks) {
    rows::combine_bwd_kernel<decltype(ty)::value, decltype(k)::value>
        <<<blocks, rows::kThreads, 0, s>>>(a);
  });
}

}  // namespace ctr

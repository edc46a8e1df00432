// gated_scan.inl -- a gated linear recurrence over packed sequences, its gradients, and one step
// of it.  Part of the translation unit of fused.hip.
//
// Sequence b has the rows [offsets[b], offsets[b + 1]).  In it, for every channel,
//   f_t = sigmoid(g_t),   h_t = f_t h_{t-1} + (1 - f_t) v_t,   h before the first row = h0[b]
//   y_t = h_t, or h_t * o_t sigmoid(o_t) with an output gate o
// and backwards, with q_t = dy_t (times o_t sigmoid(o_t)),
//   dh_t = q_t + f_{t+1} dh_{t+1} (after the last row: + dhN[b]),   dh0[b] = f_1 dh_1
//   dv_t = (1 - f_t) dh_t,   dg_t = dh_t (h_{t-1} - v_t) f_t (1 - f_t)
//   do_t = dy_t h_t sigmoid(o_t) (1 + o_t (1 - sigmoid(o_t)))
// States and gradients of them are fp32.
//
// Both directions are one long scan of affine maps h -> A h + H down all rows, A between 0 and 1.
// A map in which a sequence begins takes nothing over from before, not even an infinity times
// zero: its A has its sign bit set (-1 where a sequence begins, which products keep).  The rows are cut into chunks of kChunk, whose maps
// are made side by side, joined, and applied: work for the whole chip however few sequences and
// channels there are.
namespace ctr {
namespace scan {

constexpr int kRows = 16, kWaves = 8, kChunk = kRows * kWaves;  // rows a wave, waves a block
constexpr int kThreads = kWaves * 64;

struct Args {
  const void* g;
  int64_t gs;
  const void* v;
  int64_t vs;
  const void* o;                // nullable
  int64_t os;
  const int64_t* offsets;
  int64_t n, B;
  int D;
  const float* h0;              // nullable: 0
  void* y;
  int64_t ys;
  float* hN;                    // nullable
  float* states;                // [chunks, D]: the state before each chunk
  float* A;                     // [chunks, D]: the chunks' maps
  float* H;
  // backward
  const void* dy;
  int64_t dys;
  const float* dhN;             // nullable: 0
  void* dg;
  int64_t dgs;
  void* dv;
  int64_t dvs;
  void* dout;
  int64_t dos;
  float* dh0;                   // nullable
  float* carries;               // [chunks, D]: f dh of the row after each chunk
};

// 1 / (1 + exp(-x)) and 1 / (1 + exp(x)), each to a few units of its last place.
template <int TY>
__device__ __forceinline__ void sigmoids(float x, float* up, float* down) {
  float e, r;
  if constexpr (TY == kEltF32) {
    e = expf(-fabsf(x));
    r = 1.f / (1.f + e);
  } else {                      // inputs of 16 bits: the instructions' own exponential and inverse
    e = __expf(-fabsf(x));
    r = __builtin_amdgcn_rcpf(1.f + e);
  }
  const float s = e * r;
  *up = x >= 0.f ? r : x < 0.f ? s : x;        // NaN stays
  *down = x >= 0.f ? s : x < 0.f ? r : x;
}

__device__ __forceinline__ int64_t first_row(const Args& a) {
  return a.B > 0 ? clamp64(a.offsets[0], 0, a.n) : a.n;
}
__device__ __forceinline__ int64_t end_row(const Args& a) {
  return a.B > 0 ? clamp64(a.offsets[a.B], 0, a.n) : 0;
}

// The last sequence of those in [0, B) that begin at or before row p, 64 probes at a time; -1:
// none does.  The same in the whole wave.
__device__ __forceinline__ int64_t sequence_of(const Args& a, int64_t p) {
  const int lane = threadIdx.x & 63;
  int64_t lo = -1, hi = a.B;                   // offsets[lo] <= p < offsets[hi]
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 64) / 65;  // probes lo + step, lo + 2 step, ..
    const int64_t at = lo + (lane + 1) * step;
    const uint64_t le = __ballot(at < hi && a.offsets[at < hi ? at : hi - 1] <= p);
    const int below = le == ~0ull ? 64 : __builtin_ctzll(~le);
    const int64_t to = lo + (below + 1) * step;
    lo += below * step;
    hi = to < hi ? to : hi;
  }
  return lo;
}

// What a wave knows of its rows [p, p + kRows): which of them are in a sequence, begin one or
// end one, and the sequence of the first.
struct Marks {
  int64_t seq;                  // of row p (or -1)
  uint32_t in, begins, ends;    // bits
};
// Sequence of row i of the wave, m.seq or a later one.
__device__ __forceinline__ int64_t sequence_at(const Args& a, const Marks& m, int64_t p, int i) {
  for (int64_t b = m.seq; b < m.seq + 2; ++b)
    if (b + 1 >= a.B || a.offsets[b + 1] > p + i) return b < a.B ? b : a.B - 1;
  return sequence_of(a, p + i);
}

__device__ __forceinline__ Marks marks_of(const Args& a, int64_t p) {
  Marks m;
  m.in = m.begins = m.ends = 0u;
  const int64_t lo = first_row(a), hi = end_row(a);
  m.seq = -1;
  if (p >= hi || p + kRows <= lo) return m;
  m.seq = sequence_of(a, p);
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < kRows; ++i) m.in |= (p + i >= lo && p + i < hi ? 1u : 0u) << i;
  // offsets that lie in (p, p + kRows]: bit i of `at` is set where a sequence begins at row i
  uint32_t at = m.seq >= 0 && a.offsets[m.seq] == p ? 1u : 0u;
  for (int64_t b0 = m.seq + 1; b0 <= a.B; b0 += 64) {
    const int64_t b = b0 + lane;
    const int64_t off = b <= a.B ? a.offsets[b] : INT64_MAX;
    uint32_t mine = off > p && off <= p + kRows ? 1u << (int)(off - p) : off == p ? 1u : 0u;
    for (int d = 1; d < 64; d <<= 1) mine |= __shfl_xor(mine, d);
    at |= mine;
    if (__ballot(off > p + kRows)) break;
  }
  at = __builtin_amdgcn_readfirstlane(at);
  m.in = __builtin_amdgcn_readfirstlane(m.in);
  m.begins = at & m.in;
  m.ends = (at >> 1) & m.in;
  return m;
}

// The wave's runs of VW channels of its rows; rows outside every sequence are zeros.
template <int TY, int VW>
__device__ __forceinline__ void load_rows(Run<TY, VW> (&x)[kRows], const void* p, int64_t stride,
                                          int64_t row, uint32_t in, int c, int D) {
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    x[i].load_some(p, (row + i) * stride + c, in >> i & 1u ? D - c : 0);
}

// A map applied to what comes in.
__device__ __forceinline__ float map_on(float A, float H, float h) {
  return __float_as_uint(A) >> 31 ? H : A * h + H;
}

// The maps of all waves of a block: of those before wave w (in the scan's direction), and of all.
template <int VW>
struct Joined {
  float A[VW], H[VW], allA[VW], allH[VW];
};
template <int VW, bool BACK>
__device__ __forceinline__ Joined<VW> join_waves(float (*room)[2][64 * VW], const float* A,
                                                 const float* H) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    room[w][0][e * 64 + lane] = A[e];
    room[w][1][e * 64 + lane] = H[e];
  }
  __syncthreads();
  Joined<VW> j;
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    float pa = 1.f, ph = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const int u = BACK ? kWaves - 1 - i : i;
      if (u == w) {
        j.A[e] = pa;
        j.H[e] = ph;
      }
      const float ua = room[u][0][e * 64 + lane], uh = room[u][1][e * 64 + lane];
      ph = map_on(ua, uh, ph);
      pa = __float_as_uint(ua) >> 31 ? ua : ua * pa;
    }
    j.allA[e] = pa;
    j.allH[e] = ph;
  }
  return j;
}

// APPLY false: the chunks' maps into a.A and a.H.  true: from the states before the chunks the
// rows' results.
template <int TY, int VW, bool OUT, bool APPLY>
__global__ __launch_bounds__(kThreads) void fwd_kernel(Args a) {
  __shared__ float room[kWaves][2][64 * VW];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t chunk = blockIdx.x;
  const int c = ((int)blockIdx.y * 64 + lane) * VW;
  const int64_t p = chunk * kChunk + w * kRows;
  const Marks m = marks_of(a, p);
  Run<TY, VW> g[kRows], v[kRows], o[OUT && APPLY ? kRows : 1];
  load_rows<TY, VW>(g, a.g, a.gs, p, m.in, c, a.D);
  load_rows<TY, VW>(v, a.v, a.vs, p, m.in, c, a.D);
  if constexpr (OUT && APPLY) load_rows<TY, VW>(o, a.o, a.os, p, m.in, c, a.D);
  float A[VW], H[VW], start[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    A[e] = 1.f;
    H[e] = 0.f;
  }
  // the state that a sequence begins with
  auto begin = [&](int i) {
    const int64_t b = sequence_at(a, m, p, i);
#pragma unroll
    for (int e = 0; e < VW; ++e)
      start[e] = a.h0 && b >= 0 && c + e < a.D ? a.h0[b * a.D + c + e] : 0.f;
  };
  float f[kRows][VW], x[kRows][VW];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (!(m.in >> i & 1u)) continue;
    if (m.begins >> i & 1u) {
      begin(i);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        A[e] = -1.f;
        H[e] = start[e];
      }
    }
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float down;
      sigmoids<TY>(g[i].at(e), &f[i][e], &down);
      x[i][e] = down * v[i].at(e);
      A[e] *= f[i][e];
      H[e] = f[i][e] * H[e] + x[i][e];
    }
  }
  const Joined<VW> j = join_waves<VW, false>(room, A, H);
  if constexpr (!APPLY) {
    if (w == 0)
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (c + e < a.D) {
          a.A[chunk * a.D + c + e] = j.allA[e];
          a.H[chunk * a.D + c + e] = j.allH[e];
        }
  } else {
    float h[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const float s = c + e < a.D ? a.states[chunk * a.D + c + e] : 0.f;
      h[e] = map_on(j.A[e], j.H[e], s);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (!(m.in >> i & 1u)) continue;
      if (m.begins >> i & 1u) {
        begin(i);
#pragma unroll
        for (int e = 0; e < VW; ++e) h[e] = start[e];
      }
      float y[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        h[e] = f[i][e] * h[e] + x[i][e];
        y[e] = h[e];
        if constexpr (OUT) {
          float up, down;
          const float z = o[i].at(e);
          sigmoids<TY>(z, &up, &down);
          y[e] *= z * up;
        }
      }
      store_some<TY, VW>(a.y, (p + i) * a.ys + c, y, a.D - c);
      if (a.hN && (m.ends >> i & 1u)) {
        const int64_t b = sequence_at(a, m, p, i);
#pragma unroll
        for (int e = 0; e < VW; ++e)
          if (b >= 0 && c + e < a.D) a.hN[b * a.D + c + e] = h[e];
      }
    }
  }
}

// Backwards.  APPLY false: the maps of the chunks, from their last row to their first.  true: the
// gradients, from the states before the chunks and the carries into them from behind.
template <int TY, int VW, bool OUT, bool APPLY>
__global__ __launch_bounds__(kThreads) void bwd_kernel(Args a) {
  __shared__ float room[2][kWaves][2][64 * VW];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t chunk = blockIdx.x;
  const int c = ((int)blockIdx.y * 64 + lane) * VW;
  const int64_t p = chunk * kChunk + w * kRows;
  const Marks m = marks_of(a, p);
  Run<TY, VW> g[kRows], v[APPLY ? kRows : 1], o[OUT ? kRows : 1], dy[kRows];
  load_rows<TY, VW>(g, a.g, a.gs, p, m.in, c, a.D);
  load_rows<TY, VW>(dy, a.dy, a.dys, p, m.in, c, a.D);
  if constexpr (OUT) load_rows<TY, VW>(o, a.o, a.os, p, m.in, c, a.D);
  if constexpr (APPLY) load_rows<TY, VW>(v, a.v, a.vs, p, m.in, c, a.D);
  // row of h0, dhN or dh0 of the sequence of row i
  auto row = [&](const float* q, int i, float* x) {
    const int64_t b = sequence_at(a, m, p, i);
#pragma unroll
    for (int e = 0; e < VW; ++e) x[e] = q && b >= 0 && c + e < a.D ? q[b * a.D + c + e] : 0.f;
  };
  float before[kRows][VW];                     // the state before each row
  float A[VW], H[VW], x[VW];
  if constexpr (APPLY) {
    // forwards again: the states within the chunk
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      A[e] = 1.f;
      H[e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (!(m.in >> i & 1u)) continue;
      if (m.begins >> i & 1u) {
        row(a.h0, i, H);
#pragma unroll
        for (int e = 0; e < VW; ++e) A[e] = -1.f;
      }
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        float up, down;
        sigmoids<TY>(g[i].at(e), &up, &down);
        A[e] *= up;
        H[e] = up * H[e] + down * v[i].at(e);
      }
    }
    const Joined<VW> j = join_waves<VW, false>(room[0], A, H);
    float h[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const float s = c + e < a.D ? a.states[chunk * a.D + c + e] : 0.f;
      h[e] = map_on(j.A[e], j.H[e], s);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (m.begins >> i & 1u) row(a.h0, i, h);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        before[i][e] = h[e];
        float up, down;
        sigmoids<TY>(g[i].at(e), &up, &down);
        if (m.in >> i & 1u) h[e] = up * h[e] + down * v[i].at(e);
      }
    }
  }
  // backwards: a map takes f dh of the row behind to f dh of the first row
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    A[e] = 1.f;
    H[e] = 0.f;
  }
#pragma unroll
  for (int i = kRows - 1; i >= 0; --i) {
    if (!(m.in >> i & 1u)) continue;
    if (m.ends >> i & 1u) {
      row(a.dhN, i, H);
#pragma unroll
      for (int e = 0; e < VW; ++e) A[e] = -1.f;
    }
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float up, down, q = dy[i].at(e);
      if constexpr (OUT) {
        float zu, zd;
        const float z = o[i].at(e);
        sigmoids<TY>(z, &zu, &zd);
        q *= z * zu;
      }
      sigmoids<TY>(g[i].at(e), &up, &down);
      A[e] *= up;
      H[e] = up * (q + H[e]);
    }
  }
  const Joined<VW> j = join_waves<VW, true>(room[1], A, H);
  if constexpr (!APPLY) {
    if (w == 0)
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (c + e < a.D) {
          a.A[chunk * a.D + c + e] = j.allA[e];
          a.H[chunk * a.D + c + e] = j.allH[e];
        }
  } else {
    float carry[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const float s = c + e < a.D ? a.carries[chunk * a.D + c + e] : 0.f;
      carry[e] = map_on(j.A[e], j.H[e], s);
    }
#pragma unroll
    for (int i = kRows - 1; i >= 0; --i) {
      if (!(m.in >> i & 1u)) continue;
      if (m.ends >> i & 1u) row(a.dhN, i, carry);
      float dg[VW], dv[VW], dz[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        float up, down, q = dy[i].at(e);
        sigmoids<TY>(g[i].at(e), &up, &down);
        const float val = v[i].at(e);
        if constexpr (OUT) {
          float zu, zd;
          const float z = o[i].at(e), h = up * before[i][e] + down * val;
          sigmoids<TY>(z, &zu, &zd);
          dz[e] = q * h * zu * (1.f + z * zd);
          q *= z * zu;
        }
        const float dh = q + carry[e];
        dv[e] = down * dh;
        dg[e] = dh * (before[i][e] - val) * (up * down);
        carry[e] = up * dh;
      }
      store_some<TY, VW>(a.dv, (p + i) * a.dvs + c, dv, a.D - c);
      store_some<TY, VW>(a.dg, (p + i) * a.dgs + c, dg, a.D - c);
      if constexpr (OUT) store_some<TY, VW>(a.dout, (p + i) * a.dos + c, dz, a.D - c);
      if (a.dh0 && (m.begins >> i & 1u)) {
        const int64_t b = sequence_at(a, m, p, i);
#pragma unroll
        for (int e = 0; e < VW; ++e)
          if (b >= 0 && c + e < a.D) a.dh0[b * a.D + c + e] = carry[e];
      }
    }
  }
}

// The chunks' maps one after the other (BACK: the last first): what comes into each.
template <bool BACK>
__global__ __launch_bounds__(64) void carry_kernel(const float* __restrict__ A,
                                                   const float* __restrict__ H, int64_t chunks,
                                                   int D, float* __restrict__ into) {
  const int c = (int)blockIdx.x * 64 + threadIdx.x;
  if (c >= D) return;
  float s = 0.f;
  constexpr int DEEP = 8;
  for (int64_t i = 0; i < chunks; i += DEEP) {
    float x[DEEP], y[DEEP];
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      const int64_t at = (BACK ? chunks - 1 - i - k : i + k) * D + c;
      x[k] = i + k < chunks ? A[at] : 1.f;
      y[k] = i + k < chunks ? H[at] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      if (i + k < chunks) into[(BACK ? chunks - 1 - i - k : i + k) * D + c] = s;
      s = map_on(x[k], y[k], s);
    }
  }
}

// Sequences without rows: their states, or the gradients of them, go through.
__global__ __launch_bounds__(256) void empty_kernel(const int64_t* __restrict__ offsets, int64_t n,
                                                    int64_t B, int D,
                                                    const float* __restrict__ from,
                                                    float* __restrict__ to) {
  for (int64_t b = blockIdx.x; b < B; b += gridDim.x) {
    if (offsets[b + 1] > offsets[b]) continue;
    for (int c = threadIdx.x; c < D; c += 256) to[b * D + c] = from ? from[b * D + c] : 0.f;
  }
}

// ---------------------------------------------------------------------------------- one step
// Row i of B takes the state of slot index[i] (or i) one row further.  Rows of one slot follow each
// other in their order: the first of them takes the others along, from registers.
template <int TY, int VW, bool OUT>
__global__ __launch_bounds__(256) void step_kernel(Args a, const int32_t* __restrict__ index,
                                                   int64_t slots, const float* __restrict__ state,
                                                   float* __restrict__ next, int tiles) {
  const int64_t i = blockIdx.x / (unsigned)tiles;
  const int c = ((int)(blockIdx.x % (unsigned)tiles) * 256 + threadIdx.x) * VW;
  int64_t slot = i;
  if (index) {
    slot = index[i];
    bool seen = false;
    for (int64_t k = threadIdx.x; k < i; k += 256) seen |= index[k] == slot;
    if (__syncthreads_or(seen)) return;
  }
  const bool known = slot >= 0 && slot < slots;
  float h[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) h[e] = known && c + e < a.D ? state[slot * a.D + c + e] : 0.f;
  for (int64_t r = i; r < a.B; ++r) {
    if (r > i) {
      if (!index) break;
      // the next row of this slot
      int64_t at = a.B;
      for (int64_t k = r + threadIdx.x; k < a.B && at == a.B; k += 256)
        if (index[k] == slot) at = k;
      __shared__ unsigned long long least;
      __syncthreads();
      if (threadIdx.x == 0) least = (unsigned long long)a.B;
      __syncthreads();
      if (at < a.B) atomicMin(&least, (unsigned long long)at);
      __syncthreads();
      r = (int64_t)least;
      if (r >= a.B) break;
    }
    Run<TY, VW> g, v, o;
    g.load_some(a.g, r * a.gs + c, a.D - c);
    v.load_some(a.v, r * a.vs + c, a.D - c);
    if constexpr (OUT) o.load_some(a.o, r * a.os + c, a.D - c);
    float y[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float up, down;
      sigmoids<TY>(g.at(e), &up, &down);
      const float s = up * h[e] + down * v.at(e);
      h[e] = s;
      y[e] = s;
      if constexpr (OUT) {
        float zu, zd;
        sigmoids<TY>(o.at(e), &zu, &zd);
        y[e] *= o.at(e) * zu;
      }
      if (!known) y[e] = 0.f;
    }
    store_some<TY, VW>(a.y, r * a.ys + c, y, a.D - c);
  }
  if (known)
#pragma unroll
    for (int e = 0; e < VW; ++e)
      if (c + e < a.D) next[slot * a.D + c + e] = h[e];
}

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

// Two channels a lane where every row begins on 4 bytes (any row of binary32 does).
bool pairs(int dtype, const void* p, int64_t stride) {
  return dtype == kEltF32 ||
         (reinterpret_cast<uintptr_t>(p) % 4 == 0 && stride % 2 == 0);
}

template <int TY, bool APPLY>
void launch_fwd(const Args& a, bool two, hipStream_t s) {
  const int64_t chunks = chunks_of(a.n);
  auto go = [&](auto vw, auto out) {
    constexpr int VW = decltype(vw)::value;
    const dim3 grid((unsigned)chunks, (unsigned)((a.D + 64 * VW - 1) / (64 * VW)));
    fwd_kernel<TY, VW, decltype(out)::value, APPLY><<<grid, kThreads, 0, s>>>(a);
  };
  auto by_out = [&](auto vw) { a.o ? go(vw, std::true_type{}) : go(vw, std::false_type{}); };
  two ? by_out(std::integral_constant<int, 2>{}) : by_out(std::integral_constant<int, 1>{});
}
template <int TY, bool APPLY>
void launch_bwd(const Args& a, bool two, hipStream_t s) {
  const int64_t chunks = chunks_of(a.n);
  auto go = [&](auto vw, auto out) {
    constexpr int VW = decltype(vw)::value;
    const dim3 grid((unsigned)chunks, (unsigned)((a.D + 64 * VW - 1) / (64 * VW)));
    bwd_kernel<TY, VW, decltype(out)::value, APPLY><<<grid, kThreads, 0, s>>>(a);
  };
  auto by_out = [&](auto vw) { a.o ? go(vw, std::true_type{}) : go(vw, std::false_type{}); };
  two ? by_out(std::integral_constant<int, 2>{}) : by_out(std::integral_constant<int, 1>{});
}

unsigned empty_blocks(int64_t B) { return (unsigned)(B < 1024 ? B : 1024); }

}  // namespace scan

int64_t gated_scan_chunks(int64_t n) { return scan::chunks_of(n); }
size_t gated_scan_fwd_workspace_bytes(int64_t n, int D) {
  return 3 * (size_t)scan::chunks_of(n) * (size_t)D * 4 + 256;
}
size_t gated_scan_bwd_workspace_bytes(int64_t n, int D) {
  return 3 * (size_t)scan::chunks_of(n) * (size_t)D * 4 + 256;
}

hipError_t launch_gated_scan_fwd(const void* g, int64_t gs, const void* v, int64_t vs,
                                 const void* o, int64_t os, int dtype, const int64_t* offsets,
                                 int64_t n, int64_t B, int D, const float* h0, void* y, int64_t ys,
                                 float* hN, float* states, void* workspace, hipStream_t s) {
  scan::Args a{};
  a.g = g; a.gs = gs; a.v = v; a.vs = vs; a.o = o; a.os = os; a.offsets = offsets;
  a.n = n; a.B = B; a.D = D; a.h0 = h0; a.y = y; a.ys = ys; a.hN = hN;
  const int64_t chunks = scan::chunks_of(n), each = chunks * D;
  a.A = static_cast<float*>(workspace);
  a.H = a.A + each;
  a.states = states ? states : a.H + each;
  if (hN && B > 0)
    scan::empty_kernel<<<scan::empty_blocks(B), 256, 0, s>>>(offsets, n, B, D, h0, hN);
  if (n > 0 && B > 0) {
    const bool two = scan::pairs(dtype, g, gs) && scan::pairs(dtype, v, vs) &&
                     scan::pairs(dtype, o, os) && scan::pairs(dtype, y, ys);
    for_type(dtype, [&](auto ty) {
      constexpr int TY = decltype(ty)::value;
      scan::launch_fwd<TY, false>(a, two, s);
      scan::carry_kernel<false><<<(unsigned)((D + 63) / 64), 64, 0, s>>>(a.A, a.H, chunks, D,
                                                                         a.states);
      scan::launch_fwd<TY, true>(a, two, s);
      return hipSuccess;
    });
  }
  return hipGetLastError();
}

hipError_t launch_gated_scan_bwd(const void* g, int64_t gs, const void* v, int64_t vs,
                                 const void* o, int64_t os, int dtype, const int64_t* offsets,
                                 int64_t n, int64_t B, int D, const float* h0, const float* states,
                                 const void* dy, int64_t dys, const float* dhN, void* dg,
                                 int64_t dgs, void* dv, int64_t dvs, void* dout, int64_t dos,
                                 float* dh0, void* workspace, hipStream_t s) {
  scan::Args a{};
  a.g = g; a.gs = gs; a.v = v; a.vs = vs; a.o = o; a.os = os; a.offsets = offsets;
  a.n = n; a.B = B; a.D = D; a.h0 = h0; a.states = const_cast<float*>(states);
  a.dy = dy; a.dys = dys; a.dhN = dhN; a.dg = dg; a.dgs = dgs; a.dv = dv; a.dvs = dvs;
  a.dout = dout; a.dos = dos; a.dh0 = dh0;
  const int64_t chunks = scan::chunks_of(n), each = chunks * D;
  a.A = static_cast<float*>(workspace);
  a.H = a.A + each;
  a.carries = a.H + each;
  if (dh0 && B > 0)
    scan::empty_kernel<<<scan::empty_blocks(B), 256, 0, s>>>(offsets, n, B, D, dhN, dh0);
  if (n > 0 && B > 0) {
    const bool two = scan::pairs(dtype, g, gs) && scan::pairs(dtype, v, vs) &&
                     scan::pairs(dtype, o, os) && scan::pairs(dtype, dy, dys) &&
                     scan::pairs(dtype, dg, dgs) && scan::pairs(dtype, dv, dvs) &&
                     scan::pairs(dtype, dout, dos);
    for_type(dtype, [&](auto ty) {
      constexpr int TY = decltype(ty)::value;
      scan::launch_bwd<TY, false>(a, two, s);
      scan::carry_kernel<true><<<(unsigned)((D + 63) / 64), 64, 0, s>>>(a.A, a.H, chunks, D,
                                                                        a.carries);
      scan::launch_bwd<TY, true>(a, two, s);
      return hipSuccess;
    });
  }
  return hipGetLastError();
}

hipError_t launch_gated_scan_step(const void* g, int64_t gs, const void* v, int64_t vs,
                                  const void* o, int64_t os, int dtype, int64_t B, int D,
                                  const int32_t* index, int64_t slots, const float* state,
                                  float* next, void* y, int64_t ys, hipStream_t s) {
  if (B == 0) return hipSuccess;
  scan::Args a{};
  a.g = g; a.gs = gs; a.v = v; a.vs = vs; a.o = o; a.os = os; a.B = B; a.D = D; a.y = y; a.ys = ys;
  const bool two = scan::pairs(dtype, g, gs) && scan::pairs(dtype, v, vs) &&
                   scan::pairs(dtype, o, os) && scan::pairs(dtype, y, ys);
  return for_type(dtype, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    auto go = [&](auto vw, auto out) {
      constexpr int VW = decltype(vw)::value;
      const int tiles = (D + 256 * VW - 1) / (256 * VW);
      scan::step_kernel<TY, VW, decltype(out)::value>
          <<<(unsigned)(B * tiles), 256, 0, s>>>(a, index, slots, state, next, tiles);
    };
    auto by_out = [&](auto vw) { o ? go(vw, std::true_type{}) : go(vw, std::false_type{}); };
    two ? by_out(std::integral_constant<int, 2>{}) : by_out(std::integral_constant<int, 1>{});
    return hipGetLastError();
  });
}

}  // namespace ctr

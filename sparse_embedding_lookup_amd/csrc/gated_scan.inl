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
// zero: its A has its sign bit set (-1 where a sequence begins, which products keep).
//
// The rows are cut into chunks; a block has one chunk of 64 or 128 channels, a wave some rows of
// it, which it reads once and keeps in registers.  The block joins its waves' maps, leaves the
// chunk's map for those behind it, looks back over the chunks before it for the state that comes
// in, leaves the state that goes out, and finishes its rows.  Blocks take their chunks by a
// counter, in order: who is waited for has begun, and waits for none behind it, so every wait ends.
// What a block leaves is one 64-bit word a channel, map and all, so that no word has to be ordered
// with another.
namespace ctr {
namespace scan {

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kGroup = 16;                     // rows that one entry of marks tells of
constexpr int kFwdRows = 16, kBwdRows = 8;     // rows a wave
constexpr int kFwdChunk = kFwdRows * kWaves, kBwdChunk = kBwdRows * kWaves;
// The backward takes the state before each of its chunks from the forward.
static_assert(kFwdChunk % kBwdChunk == 0 && kBwdChunk % kFwdRows == 0, "states at whole waves");

// Of kGroup rows: the last sequence that begins at or before the first of them (-1: none), which
// rows are in a sequence, begin one, end one.
struct Marks {
  int32_t seq;
  uint16_t in, begins, ends, pad;
};

struct Args {
  const void* g;
  int64_t gs;
  const void* v;
  int64_t vs;
  const void* o;                // nullable
  int64_t os;
  const int64_t* offsets;
  int64_t n, B;
  int D, tiles;
  const float* h0;              // nullable: 0
  void* y;
  int64_t ys;
  float* hN;                    // nullable
  float* states;                // [rows / kBwdChunk, D]: the state before each chunk
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
  // workspace
  uint32_t* ticket;
  Marks* marks;                 // [rows / kGroup]
  unsigned long long* words;    // [chunks, D]
  int64_t chunks;
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

// The last sequence of those in [0, B) that begin at or before row p; -1: none does.
__device__ __forceinline__ int64_t sequence_of(const Args& a, int64_t p) {
  int64_t lo = -1, hi = a.B;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= p) lo = mid;
    else hi = mid;
  }
  return lo;
}
// Sequence of row p, m.seq or a later one; at least 0, as it indexes arrays.
__device__ __forceinline__ int64_t sequence_at(const Args& a, const Marks& m, int64_t p) {
  int64_t b = m.seq;
  for (int k = 0; k < 2; ++k, ++b)
    if (b + 1 >= a.B || a.offsets[b + 1] > p) return b < 0 ? 0 : b < a.B ? b : a.B - 1;
  b = sequence_of(a, p);
  return b < 0 ? 0 : b;
}

// Before a scan: the counter and the words cleared, the marks made, and the states (or gradients
// of them) of sequences without rows taken through.
constexpr unsigned long long kEmpty = ~0ull;   // a word that nobody has written
__global__ __launch_bounds__(256) void prepare_kernel(Args a, const float* __restrict__ from,
                                                      float* __restrict__ to) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  if (t == 0) *a.ticket = 0u;
  for (int64_t i = t; i < a.chunks * a.D; i += step) a.words[i] = kEmpty;
  const int64_t groups = (a.n + kGroup - 1) / kGroup;
  const int64_t lo = clamp64(a.offsets[0], 0, a.n), hi = clamp64(a.offsets[a.B], 0, a.n);
  for (int64_t i = t; i < groups; i += step) {
    const int64_t p = i * kGroup;
    uint32_t in = 0u, at = 0u;                 // bit q of `at`: a sequence (or their end) at p + q
    for (int q = 0; q < kGroup; ++q) in |= (p + q >= lo && p + q < hi ? 1u : 0u) << q;
    int64_t b = sequence_of(a, p);
    const int64_t seq = b;
    if (b >= 0 && a.offsets[b] == p) at |= 1u;
    // the next sequences, from one place where some begin to the next (B: the end of them)
    for (int k = 0; k <= kGroup && b < a.B; ++k) {
      const int64_t off = a.offsets[b + 1];
      if (off > p + kGroup) break;
      if (off >= p) at |= 1u << (int)(off - p);
      b = b + 2 <= a.B && a.offsets[b + 2] > off ? b + 1 : off > p ? sequence_of(a, off) : b + 1;
    }
    Marks m;
    m.seq = (int32_t)seq;
    m.in = (uint16_t)in;
    m.begins = (uint16_t)(at & in);
    m.ends = (uint16_t)((at >> 1) & in);
    m.pad = 0;
    a.marks[i] = m;
  }
  if (!to) return;
  for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (a.offsets[b + 1] > a.offsets[b]) continue;
    for (int c = threadIdx.x; c < a.D; c += 256) to[b * a.D + c] = from ? from[b * a.D + c] : 0.f;
  }
}

// Marks of the ROWS rows from p on, the same in the whole wave.
template <int ROWS>
__device__ __forceinline__ Marks marks_of(const Args& a, int64_t p) {
  Marks m{-1, 0, 0, 0, 0};
  if (p >= a.n) return m;
  m = a.marks[p / kGroup];
  const int by = (int)(p % kGroup);
  m.seq = __builtin_amdgcn_readfirstlane(m.seq);
  const uint32_t mask = (1u << ROWS) - 1u;
  m.in = (uint16_t)__builtin_amdgcn_readfirstlane((m.in >> by) & mask);
  m.begins = (uint16_t)__builtin_amdgcn_readfirstlane((m.begins >> by) & mask);
  m.ends = (uint16_t)__builtin_amdgcn_readfirstlane((m.ends >> by) & mask);
  return m;
}

// The block's chunk and its column tile.
__device__ __forceinline__ void take_ticket(const Args& a, int64_t* chunk, int* tile) {
  __shared__ uint32_t mine;
  if (threadIdx.x == 0) mine = atomicAdd(a.ticket, 1u);
  __syncthreads();
  const uint32_t t = __builtin_amdgcn_readfirstlane(mine);
  *chunk = t / (uint32_t)a.tiles;
  *tile = (int)(t % (uint32_t)a.tiles);
}

// The wave's runs of VW channels of its rows.  (Rows outside the sequences are read and not used.)
template <int TY, int VW, int ROWS>
__device__ __forceinline__ void load_rows(Run<TY, VW> (&x)[ROWS], const void* p, int64_t stride,
                                          int64_t row, int64_t n, int c, int D) {
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    x[i].load_some(p, (row + i) * stride + c, row + i < n ? D - c : 0);
}

// A map applied to what comes in, and one map after another.
__device__ __forceinline__ bool constant(float A) { return __float_as_uint(A) >> 31; }
__device__ __forceinline__ float map_on(float A, float H, float h) {
  return constant(A) ? H : A * h + H;
}
__device__ __forceinline__ void map_after(float A, float H, float* a, float* h) {
  *h = map_on(A, H, *h);
  *a = constant(A) ? A : A * *a;
}

// The maps of all waves of a block: of those before wave w (in the scan's direction), and of all.
template <int VW>
struct Joined {
  float A[VW], H[VW], allA[VW], allH[VW];
};
template <int VW>
using Room = float[kWaves][2][64 * VW];
template <int VW, bool BACK>
__device__ __forceinline__ Joined<VW> join_waves(Room<VW>& room, const float* A, const float* H) {
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
      map_after(room[u][0][e * 64 + lane], room[u][1][e * 64 + lane], &pa, &ph);
    }
    j.allA[e] = pa;
    j.allH[e] = ph;
  }
  return j;
}

// A chunk's word: its map, later the constant map of the state that goes out of it.  The A of a
// written word is never the empty word's.
__device__ __forceinline__ void leave(unsigned long long* word, float A, float H) {
  const uint32_t a = __float_as_uint(A);
  __hip_atomic_store(word,
                     (unsigned long long)(a == 0xFFFFFFFFu ? 0x7FC00000u : a) << 32 |
                         __float_as_uint(H),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What comes into the block's chunk: wave w looks at the chunk w + 1 before it (in the scan's
// direction), then the next kWaves, until the joined maps are constant in every channel.
template <int VW, bool BACK>
__device__ __forceinline__ void look_back(const Args& a, int64_t chunk, int c, Room<VW>& room,
                                          float* state) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float A[VW], H[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    A[e] = 1.f;
    H[e] = 0.f;
  }
  for (int64_t k = 1;; k += kWaves) {
    const int64_t at = BACK ? chunk + k + w : chunk - k - w;
    const bool there = at >= 0 && at < a.chunks;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float x = -1.f, y = 0.f;                 // before the first chunk there is nothing
      if (there && c + e < a.D) {
        unsigned long long word;
        while ((word = __hip_atomic_load(a.words + at * a.D + c + e, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT)) == kEmpty)
          __builtin_amdgcn_s_sleep(1);
        x = __uint_as_float((uint32_t)(word >> 32));
        y = __uint_as_float((uint32_t)word);
      }
      room[w][0][e * 64 + lane] = x;
      room[w][1][e * 64 + lane] = y;
    }
    __syncthreads();
    bool open = false;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
#pragma unroll
      for (int u = 0; u < kWaves; ++u) {
        // A, H after the map of chunk u
        const float x = room[u][0][e * 64 + lane], y = room[u][1][e * 64 + lane];
        if (!constant(A[e])) {
          H[e] = A[e] * y + H[e];
          A[e] = constant(x) ? x : A[e] * x;
        }
      }
      open |= !constant(A[e]);
    }
    if (!__any(open)) break;                   // the same in every wave
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < VW; ++e) state[e] = H[e];
}

// The chunk's map left, the state that comes in (unless a sequence begins with it), and the state
// that goes out left.
template <int VW, bool BACK>
__device__ __forceinline__ void exchange(const Args& a, int64_t chunk, int c, bool begins,
                                         const Joined<VW>& j, Room<VW>& room, float* state) {
  unsigned long long* words = a.words + chunk * a.D + c;
  const bool mine = threadIdx.x < 64;
  if (mine)
#pragma unroll
    for (int e = 0; e < VW; ++e)
      if (c + e < a.D) leave(words + e, j.allA[e], j.allH[e]);
#pragma unroll
  for (int e = 0; e < VW; ++e) state[e] = 0.f;
  if (begins) return;                          // every map is constant then
  look_back<VW, BACK>(a, chunk, c, room, state);
  if (mine)
#pragma unroll
    for (int e = 0; e < VW; ++e)
      if (c + e < a.D && !constant(j.allA[e]))
        leave(words + e, -1.f, map_on(j.allA[e], j.allH[e], state[e]));
}

template <int TY, int VW, bool OUT>
__global__ __launch_bounds__(kThreads, 4) void fwd_kernel(Args a) {
  constexpr int ROWS = kFwdRows;
  __shared__ Room<VW> room, back;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t chunk;
  int tile;
  take_ticket(a, &chunk, &tile);
  const int c = (tile * 64 + lane) * VW;
  const int64_t p = chunk * kFwdChunk + w * ROWS;
  Run<TY, VW> g[ROWS], v[ROWS], o[OUT ? ROWS : 1];
  load_rows<TY, VW, ROWS>(g, a.g, a.gs, p, a.n, c, a.D);
  load_rows<TY, VW, ROWS>(v, a.v, a.vs, p, a.n, c, a.D);
  if constexpr (OUT) load_rows<TY, VW, ROWS>(o, a.o, a.os, p, a.n, c, a.D);
  const Marks m = marks_of<ROWS>(a, p);
  const Marks top = marks_of<ROWS>(a, chunk * kFwdChunk);
  float A[VW], H[VW], start[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    A[e] = 1.f;
    H[e] = 0.f;
  }
  // the state that a sequence begins with
  auto begin = [&](int i) {
    const int64_t b = a.h0 ? sequence_at(a, m, p + i) : 0;
#pragma unroll
    for (int e = 0; e < VW; ++e) start[e] = a.h0 && c + e < a.D ? a.h0[b * a.D + c + e] : 0.f;
  };
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (!(m.in >> i & 1)) continue;
    if (m.begins >> i & 1) {
      begin(i);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        A[e] = -1.f;
        H[e] = start[e];
      }
    }
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float up, down;
      sigmoids<TY>(g[i].at(e), &up, &down);
      A[e] *= up;
      H[e] = up * H[e] + down * v[i].at(e);
    }
  }
  const Joined<VW> j = join_waves<VW, false>(room, A, H);
  float state[VW], h[VW];
  exchange<VW, false>(a, chunk, c, top.begins & 1, j, back, state);
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    h[e] = map_on(j.A[e], j.H[e], state[e]);
    if (a.states && w * ROWS % kBwdChunk == 0 && p < a.n && c + e < a.D)
      a.states[p / kBwdChunk * a.D + c + e] = h[e];
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (!(m.in >> i & 1)) continue;
    if (m.begins >> i & 1) {
      begin(i);
#pragma unroll
      for (int e = 0; e < VW; ++e) h[e] = start[e];
    }
    float y[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float up, down;
      sigmoids<TY>(g[i].at(e), &up, &down);
      h[e] = up * h[e] + down * v[i].at(e);
      y[e] = h[e];
      if constexpr (OUT) {
        const float z = o[i].at(e);
        sigmoids<TY>(z, &up, &down);
        y[e] *= z * up;
      }
    }
    store_some<TY, VW>(a.y, (p + i) * a.ys + c, y, a.D - c);
    if (a.hN && (m.ends >> i & 1)) {
      const int64_t b = sequence_at(a, m, p + i);
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (c + e < a.D) a.hN[b * a.D + c + e] = h[e];
    }
  }
}

// Backwards: a map takes f dh of the row behind it to f dh of its first row.  The states within
// the chunk are made again from the one before it.
template <int TY, int VW, bool OUT>
__global__ __launch_bounds__(kThreads, 4) void bwd_kernel(Args a) {
  constexpr int ROWS = kBwdRows;
  __shared__ Room<VW> room[2], back;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t chunk;
  int tile;
  take_ticket(a, &chunk, &tile);
  chunk = a.chunks - 1 - chunk;
  const int c = (tile * 64 + lane) * VW;
  const int64_t p = chunk * kBwdChunk + w * ROWS;
  Run<TY, VW> g[ROWS], v[ROWS], o[OUT ? ROWS : 1], dy[ROWS];
  load_rows<TY, VW, ROWS>(g, a.g, a.gs, p, a.n, c, a.D);
  load_rows<TY, VW, ROWS>(v, a.v, a.vs, p, a.n, c, a.D);
  load_rows<TY, VW, ROWS>(dy, a.dy, a.dys, p, a.n, c, a.D);
  if constexpr (OUT) load_rows<TY, VW, ROWS>(o, a.o, a.os, p, a.n, c, a.D);
  float state[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) state[e] = c + e < a.D ? a.states[chunk * a.D + c + e] : 0.f;
  const Marks m = marks_of<ROWS>(a, p);
  const int64_t final_row = chunk * kBwdChunk + kBwdChunk - ROWS;
  const Marks bottom = marks_of<ROWS>(a, final_row);
  // row of h0 or dhN of the sequence of row i
  auto row = [&](const float* q, int i, float* x) {
    const int64_t b = q ? sequence_at(a, m, p + i) : 0;
#pragma unroll
    for (int e = 0; e < VW; ++e) x[e] = q && c + e < a.D ? q[b * a.D + c + e] : 0.f;
  };
  float A[VW], H[VW], C[VW], K[VW];            // the map forwards, and backwards
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    A[e] = C[e] = 1.f;
    H[e] = K[e] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (!(m.in >> i & 1)) continue;
    if (m.begins >> i & 1) {
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
#pragma unroll
  for (int i = ROWS - 1; i >= 0; --i) {
    if (!(m.in >> i & 1)) continue;
    if (m.ends >> i & 1) {
      row(a.dhN, i, K);
#pragma unroll
      for (int e = 0; e < VW; ++e) C[e] = -1.f;
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
      C[e] *= up;
      K[e] = up * (q + K[e]);
    }
  }
  const Joined<VW> j = join_waves<VW, true>(room[1], C, K);
  float carry[VW];
  exchange<VW, true>(a, chunk, c, bottom.ends >> (ROWS - 1) & 1, j, back, carry);
#pragma unroll
  for (int e = 0; e < VW; ++e) carry[e] = map_on(j.A[e], j.H[e], carry[e]);
  const Joined<VW> f = join_waves<VW, false>(room[0], A, H);
  float before[ROWS][VW], h[VW];               // the state before each row
#pragma unroll
  for (int e = 0; e < VW; ++e) h[e] = map_on(f.A[e], f.H[e], state[e]);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (m.begins >> i & 1) row(a.h0, i, h);
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      before[i][e] = h[e];
      float up, down;
      sigmoids<TY>(g[i].at(e), &up, &down);
      if (m.in >> i & 1) h[e] = up * h[e] + down * v[i].at(e);
    }
  }
#pragma unroll
  for (int i = ROWS - 1; i >= 0; --i) {
    if (!(m.in >> i & 1)) continue;
    if (m.ends >> i & 1) row(a.dhN, i, carry);
    float dg[VW], dv[VW], dz[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float up, down, q = dy[i].at(e);
      sigmoids<TY>(g[i].at(e), &up, &down);
      const float val = v[i].at(e);
      if constexpr (OUT) {
        float zu, zd;
        const float z = o[i].at(e), now = up * before[i][e] + down * val;
        sigmoids<TY>(z, &zu, &zd);
        dz[e] = q * now * zu * (1.f + z * zd);
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
    if (a.dh0 && (m.begins >> i & 1)) {
      const int64_t b = sequence_at(a, m, p + i);
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (c + e < a.D) a.dh0[b * a.D + c + e] = carry[e];
    }
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

int64_t pieces(int64_t n, int64_t size) { return (n + size - 1) / size; }

// Four bytes a lane: a channel of binary32, or two of 16 bits where every row begins on 4 bytes.
bool pairs(int dtype, const void* p, int64_t stride) {
  return dtype != kEltF32 && reinterpret_cast<uintptr_t>(p) % 4 == 0 && stride % 2 == 0;
}

// The workspace: counter, marks, words.
size_t carve_scan(Args* a, void* workspace, int64_t n, int D, int chunk) {
  const int64_t chunks = pieces(n, chunk);
  size_t off = 256;
  char* base = static_cast<char*>(workspace);
  const size_t marks = off;
  off += ((size_t)pieces(n, kGroup) * sizeof(Marks) + 255) / 256 * 256;
  const size_t words = off;
  off += (size_t)chunks * (size_t)D * 8;
  if (a) {
    a->chunks = chunks;
    a->ticket = reinterpret_cast<uint32_t*>(base);
    a->marks = reinterpret_cast<Marks*>(base + marks);
    a->words = reinterpret_cast<unsigned long long*>(base + words);
  }
  return off;
}

hipError_t run(Args a, int dtype, bool back, bool two, hipStream_t s) {
  if (a.B == 0) return hipSuccess;
  const float* from = back ? a.dhN : a.h0;
  float* to = back ? a.dh0 : a.hN;
  if (a.n == 0 && !to) return hipSuccess;
  const int64_t work = a.chunks * a.D > a.B ? a.chunks * a.D : a.B;
  const int64_t blocks = pieces(work, 1024);
  prepare_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, s>>>(a, from, to);
  if (a.n == 0) return hipGetLastError();
  a.tiles = (int)pieces(a.D, two ? 128 : 64);
  const unsigned grid = (unsigned)(a.chunks * a.tiles);
  return for_type(dtype, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    auto go = [&](auto vw, auto out) {
      constexpr int VW = decltype(vw)::value;
      constexpr bool OUT = decltype(out)::value;
      if (back) bwd_kernel<TY, VW, OUT><<<grid, kThreads, 0, s>>>(a);
      else fwd_kernel<TY, VW, OUT><<<grid, kThreads, 0, s>>>(a);
      return hipGetLastError();
    };
    auto by_out = [&](auto vw) {
      return a.o ? go(vw, std::true_type{}) : go(vw, std::false_type{});
    };
    if constexpr (TY != kEltF32)
      if (two) return by_out(std::integral_constant<int, 2>{});
    return by_out(std::integral_constant<int, 1>{});
  });
}

}  // namespace scan

int64_t gated_scan_chunks(int64_t n) { return scan::pieces(n, scan::kBwdChunk); }
size_t gated_scan_fwd_workspace_bytes(int64_t n, int D) {
  return scan::carve_scan(nullptr, nullptr, n, D, scan::kFwdChunk);
}
size_t gated_scan_bwd_workspace_bytes(int64_t n, int D) {
  return scan::carve_scan(nullptr, nullptr, n, D, scan::kBwdChunk);
}

hipError_t launch_gated_scan_fwd(const void* g, int64_t gs, const void* v, int64_t vs,
                                 const void* o, int64_t os, int dtype, const int64_t* offsets,
                                 int64_t n, int64_t B, int D, const float* h0, void* y, int64_t ys,
                                 float* hN, float* states, void* workspace, hipStream_t s) {
  scan::Args a{};
  a.g = g; a.gs = gs; a.v = v; a.vs = vs; a.o = o; a.os = os; a.offsets = offsets;
  a.n = n; a.B = B; a.D = D; a.h0 = h0; a.y = y; a.ys = ys; a.hN = hN; a.states = states;
  scan::carve_scan(&a, workspace, n, D, scan::kFwdChunk);
  const bool two = scan::pairs(dtype, g, gs) && scan::pairs(dtype, v, vs) &&
                   scan::pairs(dtype, o, os) && scan::pairs(dtype, y, ys);
  return scan::run(a, dtype, false, two, s);
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
  scan::carve_scan(&a, workspace, n, D, scan::kBwdChunk);
  const bool two = scan::pairs(dtype, g, gs) && scan::pairs(dtype, v, vs) &&
                   scan::pairs(dtype, o, os) && scan::pairs(dtype, dy, dys) &&
                   scan::pairs(dtype, dg, dgs) && scan::pairs(dtype, dv, dvs) &&
                   scan::pairs(dtype, dout, dos);
  return scan::run(a, dtype, true, two, s);
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
    bool done = false;
    if constexpr (TY != kEltF32)
      if (two) by_out(std::integral_constant<int, 2>{}), done = true;
    if (!done) by_out(std::integral_constant<int, 1>{});
    return hipGetLastError();
  });
}

}  // namespace ctr

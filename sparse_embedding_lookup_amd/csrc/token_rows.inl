// token_rows.inl -- rows of a table by token, scaled, and the gradient of the whole table by
// sorted tokens.  Part of the translation unit of unique.hip, some of whose device code it uses.
//
//   Y[i, :]  = scale * table[ids[i], :]                        (ids[i] < 0: zeros)
//   dT[v, :] = scale * sum over i with ids[i] == v of dY[i, :]  (fp32, rows of no token zero)
//
// Gradient: the tokens sorted by row, so that each row's terms are neighbours and are added in
// the order of their positions: the same bits in every run, no atomics.
namespace ctr {
namespace tokens {

constexpr int kThreads = 256;
constexpr uint32_t kNone = 0xFFFFFFFFu;

template <bool ID64>
__device__ __forceinline__ int64_t id_of(const void* ids, int64_t i) {
  return ID64 ? static_cast<const int64_t*>(ids)[i] : (int64_t) static_cast<const int32_t*>(ids)[i];
}

// ------------------------------------------------------------------------------ forward
// G lanes (a power of two, at most 64) take a row in runs of E elements, ROWS rows at a time, so
// that as many loads of far rows are in flight.  Bound by memory: 2^20 tokens of 10^6 bf16 rows, 128
// wide, 77 us, 0.27 GB written and as much gathered; 64 tokens of 64 fp32 2.6 us.
template <int TT, int TO, bool ID64, int ROWS>
__global__ __launch_bounds__(kThreads) void fwd_kernel(const void* __restrict__ table, int64_t V,
                                                       int D, const void* __restrict__ ids,
                                                       int64_t n, float scale,
                                                       void* __restrict__ Y, int64_t ys, int G) {
  constexpr int E = TT == kEltF32 && TO == kEltF32 ? 4 : 8;
  const int l = threadIdx.x & (G - 1);
  const int64_t i0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / G * ROWS;
  int64_t id[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) id[r] = i0 + r < n ? id_of<ID64>(ids, i0 + r) : -1;
  for (int c = l * E; c < D; c += G * E) {
    Run<TT, E> x[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const bool in = id[r] >= 0 && id[r] < V;
      x[r].load_some(table, in ? id[r] * D + c : 0, in ? D - c : 0);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (i0 + r >= n) break;
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = id[r] >= V ? qnan() : x[r].at(e) * scale;
      store_some<TO, E>(Y, (i0 + r) * ys + c, v, D - c);
    }
  }
}

// ----------------------------------------------------------------------------- gradient
// Key of a token: its row, or V (the last in order, summed nowhere).
template <bool ID64>
__device__ __forceinline__ uint32_t key_of(const void* ids, int64_t i, int64_t V) {
  const int64_t id = id_of<ID64>(ids, i);
  return (uint32_t)(id >= 0 && id < V ? id : V);
}

// Floats [begin, end) of p cleared by the blocks from `first` on.
__device__ __forceinline__ void clear(float* p, int64_t begin, int64_t end, int first) {
  p += begin;
  const int64_t count = end - begin, t = (int64_t)(blockIdx.x - first) * blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)(gridDim.x - first) * blockDim.x;
  const int64_t head = (4 - (reinterpret_cast<uintptr_t>(p) >> 2 & 3)) & 3;   // to 16 bytes
  const int64_t h = head < count ? head : count, whole = (count - h) / 4;
  float4* q = reinterpret_cast<float4*>(p + h);
  for (int64_t i = t; i < whole; i += step) q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (t < h) p[t] = 0.f;
  if (t < count - h - 4 * whole) p[h + 4 * whole + t] = 0.f;
}

// Many tokens: a stable radix sort by digits of up to kDigit bits, from the lowest.  A tile is
// kSortThreads * ITEMS tokens; a pass counts the tiles' digits, scans every digit's counts over the
// tiles (by themselves in the third launch where tiles are few) and moves the tokens.  All of it
// waits more than it moves, so every launch has blocks beside that clear a share of the gradient.
// (65536 tokens of 100003 rows, 128 wide: with the table-wide clearing first and digits of 6 bits
// in tiles of 1024 44 us up to the sums, and here 29; 2^20 tokens of 10^6 rows 154 and 124 us, of
// which the clearing alone is 82.  All of a digit's counts loaded at once in the third launch: no
// difference.)
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64, kDigit = 10;
constexpr int kBins = 1 << kDigit, kFewTiles = 64;
struct Sort {
  const void* ids;              // the first pass reads the tokens themselves
  int64_t V;
  const uint32_t* keys_in;
  const uint32_t* vals_in;
  uint32_t* keys_out;
  uint32_t* vals_out;
  int64_t n;
  int shift, bits, tiles, ld;
  uint32_t* counts;             // [bins, ld]
  uint32_t* totals;             // [bins]
  float* dT;
  int64_t clear_from, clear_to;
};
// 0: later passes; 1 and 2: the first, of 32- and 64-bit tokens.
template <int FIRST>
__device__ __forceinline__ uint32_t sort_key(const Sort& g, int64_t i) {
  if constexpr (FIRST) return key_of<FIRST == 2>(g.ids, i, g.V);
  else return g.keys_in[i];
}

template <int FIRST, int ITEMS>
__global__ __launch_bounds__(kSortThreads) void count_kernel(Sort g) {
  if ((int)blockIdx.x >= g.tiles) {
    clear(g.dT, g.clear_from, g.clear_to, g.tiles);
    return;
  }
  __shared__ uint32_t bins[kBins];
  const uint32_t mask = (1u << g.bits) - 1u;
  bins[threadIdx.x] = 0u;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kSortThreads * ITEMS;
  uint32_t key[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int64_t i = base + k * kSortThreads + threadIdx.x;
    key[k] = i < g.n ? sort_key<FIRST>(g, i) : 0u;
  }
#pragma unroll
  for (int k = 0; k < ITEMS; ++k)
    count_digit(bins, key[k] >> g.shift & mask,
                base + k * kSortThreads + threadIdx.x < g.n);
  __syncthreads();
  if (threadIdx.x <= mask) g.counts[(int64_t)threadIdx.x * g.ld + blockIdx.x] = bins[threadIdx.x];
}

// A wave a digit: its counts become the tokens of it in the tiles before each.
__global__ __launch_bounds__(kSortThreads) void scan_kernel(Sort g) {
  const int blocks = ((1 << g.bits) + kSortWaves - 1) / kSortWaves;
  if ((int)blockIdx.x >= blocks) {
    clear(g.dT, g.clear_from, g.clear_to, blocks);
    return;
  }
  const int lane = threadIdx.x & 63, d = (int)blockIdx.x * kSortWaves + (threadIdx.x >> 6);
  if (d >= 1 << g.bits) return;
  uint32_t run = 0u;
  uint32_t* row = g.counts + (int64_t)d * g.ld;
  for (int i0 = 0; i0 < g.tiles; i0 += 64) {
    const int i = i0 + lane;
    const uint32_t c = i < g.tiles ? row[i] : 0u;
    uint32_t s = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t v = __shfl_up(s, o);
      if (lane >= o) s += v;
    }
    if (i < g.tiles) row[i] = run + s - c;
    run += __shfl(s, 63);
  }
  if (lane == 0) g.totals[d] = run;
}

template <int FIRST, int ITEMS>
__global__ __launch_bounds__(kSortThreads) void move_kernel(Sort g) {
  if ((int)blockIdx.x >= g.tiles) {
    clear(g.dT, g.clear_from, g.clear_to, g.tiles);
    return;
  }
  __shared__ uint32_t waves[kSortWaves][kBins];   // tokens of a digit in a wave, then before it
  __shared__ uint32_t start[kBins], sums[kSortWaves];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, me = (int)blockIdx.x;
  const int bins = 1 << g.bits;
  const uint32_t mask = (uint32_t)bins - 1u;
  // a wave has ITEMS * 64 neighbouring tokens, in their order
  const int64_t base = (int64_t)me * kSortThreads * ITEMS + w * 64 * ITEMS;
  uint32_t key[ITEMS], val[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int64_t i = base + k * 64 + lane;
    key[k] = i < g.n ? sort_key<FIRST>(g, i) : 0u;
    val[k] = FIRST ? (uint32_t)i : i < g.n ? g.vals_in[i] : 0u;
  }
  // digit t: its tokens in all tiles, and in the tiles before this one
  uint32_t total = 0u, before = 0u;
  if (t < bins) {
    if (g.tiles <= kFewTiles) {
      const uint4* row = reinterpret_cast<const uint4*>(g.counts + (int64_t)t * g.ld);
#pragma unroll 4
      for (int q = 0; q < g.ld / 4; ++q) {
        const uint4 v = row[q];
        const uint32_t c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = 4 * q + j < g.tiles ? c[j] : 0u;
          total += x;
          before += 4 * q + j < me ? x : 0u;
        }
      }
    } else {
      total = g.totals[t];
      before = g.counts[(int64_t)t * g.ld + me];
    }
  }
  for (int i = t; i < kSortWaves * bins; i += kSortThreads) waves[i >> g.bits][i & mask] = 0u;
  uint32_t upto = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 63) sums[w] = upto;
  __syncthreads();
  for (int u = 0; u < w; ++u) upto += sums[u];
  start[t] = upto - total + before;
  // a token's place among those of its digit in the wave: by the lanes that share it
  uint64_t same[ITEMS];
  uint32_t first[ITEMS];
  const uint64_t lower = lanemask_lt();
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const bool live = base + k * 64 + lane < g.n;
    const uint32_t d = key[k] >> g.shift & mask;
    same[k] = match_digit(d, g.bits, __ballot(live));
    first[k] = 0u;
    if (live && (same[k] & lower) == 0ull)
      first[k] = atomicAdd(&waves[w][d], (uint32_t)__popcll(same[k]));
  }
  __syncthreads();
  if (t < bins) {
    uint32_t run = start[t];
#pragma unroll
    for (int u = 0; u < kSortWaves; ++u) {
      const uint32_t c = waves[u][t];
      waves[u][t] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int leader = same[k] ? (int)__builtin_ctzll(same[k]) : 0;
    const uint32_t rank = (uint32_t)__shfl((int)first[k], leader) +
                          (uint32_t)__popcll(same[k] & lower);
    if (base + k * 64 + lane < g.n) {
      const uint32_t at = waves[w][key[k] >> g.shift & mask] + rank;
      g.keys_out[at] = key[k];
      g.vals_out[at] = val[k];
    }
  }
}

// Few tokens: sorted in this launch, for a sort of several would be latency alone.  A token's place
// is the number of tokens before it in order; a block has 16 tokens and each of them 16 threads, which
// compare it with every sixteenth of all.
constexpr int kRankTile = 4096, kRankOf = 16;
template <bool ID64>
__global__ __launch_bounds__(kThreads) void rank_kernel(const void* __restrict__ ids, int n,
                                                        int64_t V, int key_blocks,
                                                        uint32_t* __restrict__ sk,
                                                        uint32_t* __restrict__ sv,
                                                        float* __restrict__ dT, int64_t count) {
  if ((int)blockIdx.x >= key_blocks) {
    clear(dT, 0, count, key_blocks);
    return;
  }
  __shared__ __attribute__((aligned(16))) uint32_t tile[kRankTile];
  const int t = threadIdx.x, i = (int)blockIdx.x * kRankOf + t / kRankOf, part = t % kRankOf;
  const uint32_t key = i < n ? key_of<ID64>(ids, i, V) : kNone;
  int before = 0;
  for (int t0 = 0; t0 < n; t0 += kRankTile) {
    const int m = n - t0 < kRankTile ? n - t0 : kRankTile;
    __syncthreads();
#pragma unroll 8
    for (int j = t; j < (m + 3) / 4 * 4; j += kThreads)
      tile[j] = j < m ? key_of<ID64>(ids, t0 + j, V) : kNone;
    __syncthreads();
#pragma unroll 4
    for (int j = 4 * part; j < m; j += 4 * kRankOf) {
      const uint4 k = *reinterpret_cast<const uint4*>(tile + j);
      const int at = i - (t0 + j);             // equal keys count where they come before
      before += (k.x < key + (at > 0)) + (k.y < key + (at > 1)) + (k.z < key + (at > 2)) +
                (k.w < key + (at > 3));
    }
  }
#pragma unroll
  for (int d = 1; d < kRankOf; d <<= 1) before += __shfl_xor(before, d);
  if (i < n && part == 0) {
    sk[before] = key;
    sv[before] = (uint32_t)i;
  }
}

// Sums of the sorted tokens' rows.  A block has 256 / G groups of G lanes, a group `chunk`
// neighbouring sorted positions and a lane E columns of them.  A group stores the sums of the
// rows that begin and end inside it; its first and its last go through LDS, where the group where
// a row begins joins what the groups after it have of it, in order.  What a block shares with its neighbours (the rows of its first and last
// position) goes to `part`, two sums a block, for join_kernel.
// Bound by the gather of dY's rows in the order of the keys: 2^20 rows of 128 bf16 131 us, 0.27 GB
// gathered and the sums written; 65536 10 us.  (Chunks of 8 to 128 positions and rows through LDS
// ahead of their use were all within 5 % of that.  With one group that joins the firsts and lasts of
// all, one after the other, 136 and 16 us, and 19 for 256 rows of 64, now 5.)
struct Sums {
  const uint32_t* sk;
  const uint32_t* sv;
  int64_t n;
  uint32_t V;
  const void* dY;
  int64_t dys;
  int D, G, chunk;
  float scale;
  float* dT;
  float* part;                  // [2 * blocks, D]: of the row that came in, of the row that goes on
  uint32_t* part_key;           // [2 * blocks], kNone: there is none
};

template <int TY>
constexpr int kSumElts = TY == kEltF32 ? 4 : 8;

template <int N>
__device__ __forceinline__ void put_sum(float* row, int c, int D, const float* s, float scale) {
  float v[N];
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = s[e] * scale;
  store_some<kEltF32, N>(row, c, v, D - c);
}

template <int TY>
__global__ __launch_bounds__(kThreads) void sum_kernel(Sums g) {
  constexpr int E = kSumElts<TY>, DEEP = 8;
  __shared__ float sums[2][kThreads * E];
  __shared__ uint32_t keys[2][kThreads];
  const int t = threadIdx.x, l = t & (g.G - 1), group = t / g.G, groups = kThreads / g.G;
  const int c = ((int)blockIdx.y * g.G + l) * E;
  const int there = c < g.D ? g.D - c : 0;
  const int64_t a = ((int64_t)blockIdx.x * groups + group) * g.chunk;
  const int64_t b = a + g.chunk < g.n ? a + g.chunk : g.n;
  // the block's positions, and the rows before and behind them
  const int64_t lo = (int64_t)blockIdx.x * groups * g.chunk, hi = lo + (int64_t)groups * g.chunk;
  const uint32_t came = lo > 0 ? g.sk[lo - 1] : kNone, goes = hi < g.n ? g.sk[hi] : kNone;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  uint32_t cur = kNone, first = kNone;
  bool head = true;
  for (int64_t p = a; p < b; p += DEEP) {
    uint32_t key[DEEP], row[DEEP];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      const bool in = p + i < b;
      key[i] = in ? g.sk[p + i] : kNone;
      row[i] = in ? g.sv[p + i] : 0u;
    }
    Run<TY, E> x[DEEP];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      const bool in = key[i] < g.V;
      x[i].load_some(g.dY, in ? (int64_t)row[i] * g.dys + c : 0, in ? there : 0);
    }
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      if (p + i >= b) break;
      if (key[i] != cur) {
        if (cur != kNone) {
          if (head) {
            first = cur;
#pragma unroll
            for (int e = 0; e < E; ++e) sums[0][e * kThreads + t] = acc[e];
            head = false;
          } else if (cur < g.V && there > 0) {
            put_sum<E>(g.dT + (int64_t)cur * g.D, c, g.D, acc, g.scale);
          }
        }
        cur = key[i];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += x[i].at(e);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sums[1][e * kThreads + t] = acc[e];
  keys[0][t] = first;
  keys[1][t] = cur;
  __syncthreads();
  // The runs of one row over the groups' firsts and lasts: each by the group where it begins.
  auto emit = [&](uint32_t run, const float* v) {
    if (run >= g.V || there <= 0) return;      // that of no token
    if (run == came) put_sum<E>(g.part + (int64_t)blockIdx.x * 2 * g.D, c, g.D, v, 1.f);
    else if (run == goes) put_sum<E>(g.part + ((int64_t)blockIdx.x * 2 + 1) * g.D, c, g.D, v, 1.f);
    else put_sum<E>(g.dT + (int64_t)run * g.D, c, g.D, v, g.scale);
  };
  const uint32_t left = group > 0 ? keys[1][t - g.G] : kNone;
  if (first != kNone && first != left) {       // and its last is another
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = sums[0][e * kThreads + t];
    emit(first, acc);
  }
  if (cur != kNone && (first != kNone || cur != left)) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = sums[1][e * kThreads + t];
    constexpr int STEP = 4;
    bool on = true;
    for (int u = group + 1; on && u < groups; u += STEP) {
      float x[STEP][E];
      bool same[STEP], whole[STEP];            // its first or all of it is of this row
#pragma unroll
      for (int i = 0; i < STEP; ++i) {
        const int at = (u + i < groups ? u + i : groups - 1) * g.G + l;
        const uint32_t head = keys[0][at];
        whole[i] = head == kNone;
        same[i] = u + i < groups && (whole[i] ? keys[1][at] : head) == cur;
        const float* from = sums[whole[i] ? 1 : 0] + at;
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] = from[e * kThreads];
      }
#pragma unroll
      for (int i = 0; i < STEP; ++i) {
        on = on && same[i];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = on ? acc[e] + x[i][e] : acc[e];
        on = on && whole[i];
      }
    }
    emit(cur, acc);
  }
  if (t == 0 && blockIdx.y == 0) {
    g.part_key[2 * blockIdx.x] = came < g.V && g.sk[lo] == came ? came : kNone;
    g.part_key[2 * blockIdx.x + 1] =
        goes < g.V && goes != came && g.sk[hi - 1] == goes ? goes : kNone;
  }
}

// The rows that several blocks share: the block where one begins adds what goes on from there
// and what came into the blocks after it, each group every 256 / G-th of them, then the groups'
// sums in order.  (Latency: 4.6 us for 512 blocks' sums, 6.1 for 2048.)
template <int E>
__global__ __launch_bounds__(kThreads) void join_kernel(Sums g, int64_t blocks) {
  __shared__ float sums[kThreads * E];
  const uint32_t key = g.part_key[2 * blockIdx.x + 1];
  if (key == kNone) return;                    // the same in the whole block
  const int t = threadIdx.x, l = t & (g.G - 1), group = t / g.G, groups = kThreads / g.G;
  const int c = ((int)blockIdx.y * g.G + l) * E;
  const int there = c < g.D ? g.D - c : 0;
  float s[E];
#pragma unroll
  for (int e = 0; e < E; ++e) s[e] = 0.f;
  constexpr int DEEP = 4;
  bool more = true;
  for (int64_t j = (int64_t)blockIdx.x + 1 + group; more && j < blocks; j += DEEP * groups) {
    Run<kEltF32, E> x[DEEP];
    bool in[DEEP];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      const int64_t k = j + i * groups;
      in[i] = k < blocks && g.part_key[2 * k] == key;
    }
#pragma unroll
    for (int i = 0; i < DEEP; ++i)
      x[i].load_some(g.part, in[i] ? 2 * (j + i * groups) * g.D + c : 0, in[i] ? there : 0);
#pragma unroll
    for (int i = 0; i < DEEP; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) s[e] += x[i].at(e);
    more = in[DEEP - 1];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sums[e * kThreads + t] = s[e];
  __syncthreads();
  if (group != 0 || there == 0) return;
  Run<kEltF32, E> x;
  x.load_some(g.part, (2 * (int64_t)blockIdx.x + 1) * g.D + c, there);
#pragma unroll
  for (int e = 0; e < E; ++e) s[e] = x.at(e);
  for (int u = 0; u < groups; ++u)
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] += sums[e * kThreads + u * g.G + l];
  put_sum<E>(g.dT + (int64_t)key * g.D, c, g.D, s, g.scale);
}

// Lanes a row of D elements in runs of E: a power of two, at most 64.
int lanes(int D, int E) {
  int G = 1;
  while (G < 64 && G * E < D) G <<= 1;
  return G;
}

// (The whole gradient, 64 wide, of 1000 and of 10^6 rows by ranks and by the sort: 1024 tokens 14 and
// 18, 43 and 48 us; 4096 19 and 19, 45 and 49; 8192 27 and 20, 48 and 49.)
constexpr int64_t kRankMost = 4096;

int key_bits(int64_t V) {
  int b = 1;
  while (V >> b) ++b;
  return b;
}

// Sorted positions a group takes: enough blocks for the chip first, then longer runs, which
// leave fewer sums to join.
int chunk_of(int64_t n, int G) {
  const int64_t groups = kThreads / G;
  int chunk = 8;
  while (chunk < 32 && n > 1024 * groups * chunk) chunk *= 2;
  return chunk;
}

struct Workspace {
  uint32_t* keys[2];
  uint32_t* vals[2];
  uint32_t* counts;
  uint32_t* totals;
  float* part;
  uint32_t* part_key;
  int64_t blocks;
  size_t bytes;
};
// Tokens a thread in a sort's tile: one until there is a tile for every compute unit, then four.
// (The whole gradient, 64 wide, of 10^6 rows: 262144 tokens 96 us with one and 103 with four, 524288
// 143 and 127.)
int sort_items(int64_t n) { return n <= (int64_t)256 * kSortThreads ? 1 : 4; }
int64_t sort_tiles(int64_t n) {
  const int64_t tile = (int64_t)kSortThreads * sort_items(n);
  return (n + tile - 1) / tile;
}
Workspace carve_tokens(void* base, int64_t n, int D, int E) {
  Workspace w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? static_cast<char*>(base) + off : nullptr;
    off += align256(bytes);
    return p;
  };
  for (int i = 0; i < 2; ++i) w.keys[i] = reinterpret_cast<uint32_t*>(take(4 * (size_t)n));
  for (int i = 0; i < 2; ++i) w.vals[i] = reinterpret_cast<uint32_t*>(take(4 * (size_t)n));
  const size_t ld = n > kRankMost ? (size_t)(sort_tiles(n) + 3) / 4 * 4 : 0;
  w.counts = reinterpret_cast<uint32_t*>(take(4 * kBins * ld));
  w.totals = reinterpret_cast<uint32_t*>(take(4 * (size_t)kBins));
  const int G = lanes(D, E);
  const int64_t each = (int64_t)(kThreads / G) * chunk_of(n, G);
  w.blocks = (n + each - 1) / each;
  w.part = reinterpret_cast<float*>(take(8 * (size_t)w.blocks * (size_t)D));
  w.part_key = reinterpret_cast<uint32_t*>(take(8 * (size_t)w.blocks));
  w.bytes = off;
  return w;
}

}  // namespace tokens

size_t token_embed_bwd_workspace_bytes(int64_t n, int D, int dtype) {
  return tokens::carve_tokens(nullptr, n, D, dtype == kEltF32 ? 4 : 8).bytes;
}

hipError_t launch_token_embed_fwd(const void* table, int dtype, int64_t V, int D, const void* ids,
                                  bool ids64, int64_t n, float scale, void* Y, int out_dtype,
                                  int64_t ys, hipStream_t s) {
  if (n == 0) return hipSuccess;
  return for_type(dtype, [&](auto tt) {
    return for_type(out_dtype, [&](auto to) {
      constexpr int TT = decltype(tt)::value, TO = decltype(to)::value;
      const int G = tokens::lanes(D, TT == kEltF32 && TO == kEltF32 ? 4 : 8);
      // one row a group until the chip is full several times over, then four (128 bf16 of 10^6 rows:
      // 4096 tokens 2.7 and 3.2 us, 65536 6.6 and 6.6, 2^20 107 and 85)
      auto launch = [&](auto id64, auto rows) {
        constexpr int R = decltype(rows)::value;
        const int64_t groups = (n + R - 1) / R, per = tokens::kThreads / G;
        tokens::fwd_kernel<TT, TO, decltype(id64)::value, R>
            <<<(unsigned)((groups + per - 1) / per), tokens::kThreads, 0, s>>>(
                table, V, D, ids, n, scale, Y, ys, G);
        return hipGetLastError();
      };
      auto by_id = [&](auto rows) {
        return ids64 ? launch(std::true_type{}, rows) : launch(std::false_type{}, rows);
      };
      return n * G < (int64_t)1 << 20 ? by_id(std::integral_constant<int, 1>{})
                                      : by_id(std::integral_constant<int, 4>{});
    });
  });
}

hipError_t launch_token_embed_bwd(const void* dY, int dtype, int64_t dys, const void* ids,
                                  bool ids64, int64_t n, int64_t V, int D, float scale, float* dT,
                                  void* workspace, hipStream_t s) {
  const int64_t count = V * D;
  const int E = dtype == kEltF32 ? 4 : 8;
  tokens::Workspace w = tokens::carve_tokens(workspace, n, D, E);
  int64_t clear = (count + 16 * tokens::kThreads - 1) / (16 * tokens::kThreads);
  if (clear > 4096) clear = 4096;
  const uint32_t* sk = w.keys[0];
  const uint32_t* sv = w.vals[0];
  if (n <= tokens::kRankMost) {
    const int kb = (int)((n + tokens::kRankOf - 1) / tokens::kRankOf);
    if (kb + clear == 0) return hipSuccess;
    if (ids64)
      tokens::rank_kernel<true><<<(unsigned)(kb + clear), tokens::kThreads, 0, s>>>(
          ids, (int)n, V, kb, w.keys[0], w.vals[0], dT, count);
    else
      tokens::rank_kernel<false><<<(unsigned)(kb + clear), tokens::kThreads, 0, s>>>(
          ids, (int)n, V, kb, w.keys[0], w.vals[0], dT, count);
  } else {
    tokens::Sort q{};
    q.ids = ids; q.V = V; q.n = n; q.dT = dT; q.counts = w.counts; q.totals = w.totals;
    const int items = tokens::sort_items(n), bits = tokens::key_bits(V);
    const int passes = (bits + tokens::kDigit - 1) / tokens::kDigit;
    q.tiles = (int)tokens::sort_tiles(n);
    q.ld = (q.tiles + 3) / 4 * 4;
    const bool scan = q.tiles > tokens::kFewTiles;
    const int launches = passes * (scan ? 3 : 2);
    int launched = 0;
    // the grid of a launch with `own` blocks of its own, and its share of the clearing
    auto grid = [&](int own) {
      q.clear_from = count / launches * launched;
      q.clear_to = ++launched == launches ? count : count / launches * launched;
      const int64_t share = q.clear_to - q.clear_from, each = 16 * tokens::kSortThreads;
      const int64_t blocks = (share + each - 1) / each;
      return (unsigned)(own + (blocks < 4096 ? blocks : 4096));
    };
    for (int p = 0; p < passes; ++p) {
      q.bits = (bits - q.shift) / (passes - p);            // spread evenly
      q.keys_out = w.keys[p & 1];
      q.vals_out = w.vals[p & 1];
      auto by_items = [&](auto kernel) {
        return items == 1 ? kernel(std::integral_constant<int, 1>{})
                          : kernel(std::integral_constant<int, 4>{});
      };
      auto by_pass = [&](auto kernel) {
        if (p > 0) kernel(std::integral_constant<int, 0>{});
        else if (ids64) kernel(std::integral_constant<int, 2>{});
        else kernel(std::integral_constant<int, 1>{});
      };
      unsigned blocks = grid(q.tiles);
      by_pass([&](auto f) {
        by_items([&](auto k) {
          tokens::count_kernel<decltype(f)::value, decltype(k)::value>
              <<<blocks, tokens::kSortThreads, 0, s>>>(q);
        });
      });
      if (scan) {
        blocks = grid(((1 << q.bits) + tokens::kSortWaves - 1) / tokens::kSortWaves);
        tokens::scan_kernel<<<blocks, tokens::kSortThreads, 0, s>>>(q);
      }
      blocks = grid(q.tiles);
      by_pass([&](auto f) {
        by_items([&](auto k) {
          tokens::move_kernel<decltype(f)::value, decltype(k)::value>
              <<<blocks, tokens::kSortThreads, 0, s>>>(q);
        });
      });
      q.shift += q.bits;
      sk = q.keys_in = q.keys_out;
      sv = q.vals_in = q.vals_out;
    }
  }
  if (n == 0) return hipGetLastError();
  tokens::Sums g{};
  g.sk = sk; g.sv = sv; g.n = n; g.V = (uint32_t)V;
  g.dY = dY; g.dys = dys; g.D = D; g.scale = scale; g.dT = dT;
  g.part = w.part; g.part_key = w.part_key;
  g.G = tokens::lanes(D, E);
  g.chunk = tokens::chunk_of(n, g.G);
  const dim3 grid((unsigned)w.blocks, (unsigned)((D + g.G * E - 1) / (g.G * E)));
  return for_type(dtype, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    tokens::sum_kernel<TY><<<grid, tokens::kThreads, 0, s>>>(g);
    tokens::join_kernel<tokens::kSumElts<TY>><<<grid, tokens::kThreads, 0, s>>>(g, w.blocks);
    return hipGetLastError();
  });
}

}  // namespace ctr

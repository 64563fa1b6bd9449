// Tokens sorted by expert and back, with the routing weights, and the
// gradient (include/mm.h, mm_moe_permute).  Assignment a = t*k + s goes to
// row pos[a] = offset[e] + (number of assignments to e before a), where
// group e starts at offset[e], a multiple of `align`; an expert index
// outside [0, E) drops the assignment (pos -1).  Each kernel reads a token's
// row once and is bound by the row traffic; the indices are small beside it.
#include "mm_kernels.cuh"
#include "pack.cuh"

namespace mm {

constexpr int kPmThreads = 512;         // sort and copy: two blocks an SM
constexpr int kPmWarps = kPmThreads / 32;
constexpr int kPmKept = 2048;           // positions of a block kept in shared memory
constexpr int kPmRowThreads = 128;      // combine and its gradient: small blocks, which even out the SMs' paces

// Calls f(row) for the padding rows of every group, shared out over the grid's
// warps (this one is w of n); the whole warp calls.  Rows are kept inside
// [0, rows) whatever the tables hold.
template <typename F>
__device__ __forceinline__ void each_padding_row(const int32_t* offsets, const int32_t* counts, int E,
                                                 int64_t rows, int64_t w, int64_t n, F&& f) {
  const int lane = threadIdx.x & 31;
  // lane l holds groups l and l + 32: first padding row, rows before and behind it in the count
  int first[2], from[2], to[2], total = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = lane + 32 * i;
    int num = 0;
    first[i] = 0;
    if (e < E) {
      int64_t p0 = static_cast<int64_t>(offsets[e]) + counts[e], p1 = offsets[e + 1];
      p0 = p0 < 0 ? 0 : p0;
      p1 = p1 > rows ? rows : p1;
      first[i] = static_cast<int>(p0);
      num = p1 > p0 ? static_cast<int>(p1 - p0) : 0;
    }
    int sum = num;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    to[i] = total + sum;
    from[i] = to[i] - num;
    total += __shfl_sync(0xffffffffu, sum, 31);
  }
  for (int64_t p = w; p < total; p += n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const unsigned hit = __ballot_sync(0xffffffffu, p >= from[i] && p < to[i]);
      if (hit == 0) continue;
      const int src = __ffs(hit) - 1;
      f(static_cast<int64_t>(__shfl_sync(0xffffffffu, first[i], src)) + (p - __shfl_sync(0xffffffffu, from[i], src)));
    }
}
static_assert(MM_MAX_EXPERTS <= 64, "each_padding_row: two groups a lane");

// Assignments to each expert among [first, first + num) of topk_idx, added to
// cnt in shared memory (integers: any order gives the same sums).
__device__ __forceinline__ void count_experts(const int32_t* topk_idx, int64_t first, int64_t num, int E,
                                              int* cnt) {
  constexpr int kBatch = 8;                   // loads in flight a thread
  for (int64_t i0 = threadIdx.x; i0 < num; i0 += static_cast<int64_t>(blockDim.x) * kBatch) {
    int e[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int64_t i = i0 + static_cast<int64_t>(q) * blockDim.x;
      e[q] = i < num ? topk_idx[first + i] : -1;
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q)
      if (e[q] >= 0 && e[q] < E) atomicAdd(&cnt[e[q]], 1);
  }
}

// counts [block][E]: the block's assignments per expert.
__global__ void __launch_bounds__(128) permute_count_kernel(const PermuteArgs a, int tokens, int32_t* blk_cnt) {
  pdl_enter();
  __shared__ int cnt[MM_MAX_EXPERTS];
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int64_t nt = a.T - t0 < tokens ? a.T - t0 : tokens;
  count_experts(a.topk_idx, t0 * a.k, nt * a.k, a.E, cnt);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) blk_cnt[blockIdx.x * a.E + e] = cnt[e];
}

// Block b owns the assignments of `tokens` tokens from b * tokens on.  It
// works out its own base in every group - from the blocks' counts, or
// (blk_cnt null: few assignments) by counting all of them itself, which
// saves a launch - then its assignments' ranks, and (copy) copies its rows, in
// pieces shared out over its warps: one load, a store for each of the token's
// assignments.  The rows are asked for (to L2) before the indices are worked
// out.  Blocks from `owners` on own no token; they zero padding.
template <typename Vec>
__global__ void __launch_bounds__(kPmThreads, 2)
permute_kernel(const PermuteArgs a, int tokens, int owners, const int32_t* blk_cnt, int row_bytes, int copy) {
  constexpr int kBatch = sizeof(Vec) == 16 ? 4 : sizeof(Vec) == 8 ? 6 : 12;      // vectors of a row in flight a lane
  __shared__ int s_tot[MM_MAX_EXPERTS], s_next[MM_MAX_EXPERTS], s_off[MM_MAX_EXPERTS + 1];
  __shared__ int s_warp[kPmWarps][MM_MAX_EXPERTS];
  __shared__ int s_pos[kPmKept];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = static_cast<int>(blockIdx.x) < owners ? static_cast<int64_t>(blockIdx.x) * tokens : a.T;
  const int nt = static_cast<int>(a.T - t0 < tokens ? a.T - t0 : tokens), na = nt * a.k;
  const int32_t* idx = a.topk_idx + t0 * a.k;
  const char* x = static_cast<const char*>(a.x) + t0 * row_bytes;
  if (copy && nt > 0 && sizeof(Vec) == 16 && tid == 0) {
    // at most 64 KB a block: 20 MB over the grid, well inside L2
    const int64_t all = static_cast<int64_t>(nt) * row_bytes, bytes = all < 65536 ? all : 65536;
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(x), "r"(static_cast<uint32_t>(bytes)) : "memory");
  }
  for (int e = tid; e < a.E; e += kPmThreads) s_tot[e] = s_next[e] = 0;
  pdl_enter();
  const int nv = row_bytes / static_cast<int>(sizeof(Vec)), chunks = (nv + 32 * kBatch - 1) / (32 * kBatch);
  Vec v[kBatch];
  auto fetch = [&](int token, int chunk) {
    const Vec* src = reinterpret_cast<const Vec*>(x + static_cast<int64_t>(token) * row_bytes);
    const int c = chunk * (32 * kBatch) + lane;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c + 32 * i < nv) v[i] = src[c + 32 * i];
  };
  const int own = tid < na ? idx[tid] : -1;    // the first round's, on its way meanwhile
  __syncthreads();
  if (blk_cnt == nullptr) {
    count_experts(a.topk_idx, 0, t0 * a.k, a.E, s_next);
    count_experts(a.topk_idx, t0 * a.k, (a.T - t0) * a.k, a.E, s_tot);
    __syncthreads();
    for (int e = tid; e < a.E; e += kPmThreads) s_tot[e] += s_next[e];
  } else {
    // thread: one expert, every `parts`-th block
    const int e = tid % a.E, part = tid / a.E, parts = kPmThreads / a.E;
    if (part < parts) {
      int all = 0, before = 0;
      for (int b0 = part; b0 < owners; b0 += 8 * parts) {
        int c[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) c[q] = b0 + q * parts < owners ? blk_cnt[(b0 + q * parts) * a.E + e] : 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          all += c[q];
          before += b0 + q * parts < static_cast<int>(blockIdx.x) ? c[q] : 0;
        }
      }
      atomicAdd(&s_tot[e], all);              // integers: any order gives the same sums
      atomicAdd(&s_next[e], before);
    }
  }
  __syncthreads();
  if (warp == 0) {                            // offsets: a scan of the padded counts
    int run = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane, own = e < a.E ? (s_tot[e] + a.align - 1) / a.align * a.align : 0;
      int sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      if (e < a.E) {
        s_off[e] = run + sum - own;
        s_next[e] += run + sum - own;         // the block's next row in the group
      }
      run += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) s_off[a.E] = run;
  }
  __syncthreads();
  // ranks, one assignment a thread and round: within the warp, then the warps in order
  for (int base = 0; base < na; base += kPmThreads) {
    const int i = base + tid;
    const int e = base == 0 ? own : i < na ? idx[i] : -1;
    const bool valid = e >= 0 && e < a.E;
    const unsigned peers = __match_any_sync(0xffffffffu, valid ? e : -1);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    for (int q = lane; q < a.E; q += 32) s_warp[warp][q] = 0;
    __syncwarp();
    if (valid && rank == 0) s_warp[warp][e] = __popc(peers);
    __syncthreads();
    int row = -1;
    if (valid) {
      row = s_next[e] + rank;
      for (int w = 0; w < warp; ++w) row += s_warp[w][e];
    }
    if (i < na) {
      a.pos[t0 * a.k + i] = row;
      if (i < kPmKept) s_pos[i] = row;
      if (valid) a.perm[row] = static_cast<int32_t>(t0 * a.k + i);
    }
    __syncthreads();
    for (int q = tid; q < a.E; q += kPmThreads)
      for (int w = 0; w < kPmWarps; ++w) s_next[q] += s_warp[w][q];
    __syncthreads();
  }
  // rows: the next piece's load is under way while this one is stored
  int item = warp, token = item / chunks, chunk = item - token * chunks;
  const int items = copy ? nt * chunks : 0;
  if (item < items) fetch(token, chunk);
  while (item < items) {
    Vec now[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) now[i] = v[i];
    const int c = chunk * (32 * kBatch) + lane, first = token * a.k;
    item += kPmWarps;
    token = item / chunks;
    chunk = item - token * chunks;
    if (item < items) fetch(token, chunk);
    for (int at = first; at < first + a.k; ++at) {
      const int64_t row = at < kPmKept ? s_pos[at] : a.pos[t0 * a.k + at];    // the block's own writes
      if (row < 0) continue;
      Vec* dst = reinterpret_cast<Vec*>(static_cast<char*>(a.xs) + row * row_bytes);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (c + 32 * i < nv) dst[c + 32 * i] = now[i];
    }
  }
  if (blockIdx.x == 0) {
    for (int e = tid; e <= a.E; e += kPmThreads) a.offsets[e] = s_off[e];
    for (int e = tid; e < a.E; e += kPmThreads) a.counts[e] = s_tot[e];
  }
  const int64_t wg = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x, nw = static_cast<int64_t>(gridDim.x) * kPmWarps;
  if (a.align > 1)
    each_padding_row(s_off, s_tot, a.E, a.rows, wg, nw, [&](int64_t row) {
      Vec* dst = reinterpret_cast<Vec*>(static_cast<char*>(a.xs) + row * row_bytes);
      for (int c = lane; copy && c < nv; c += 32) dst[c] = Vec{};
      if (lane == 0) a.perm[row] = -1;
    });
  for (int64_t r = s_off[a.E] + static_cast<int64_t>(blockIdx.x) * kPmThreads + tid; r < a.rows;
       r += static_cast<int64_t>(gridDim.x) * kPmThreads)
    a.perm[r] = -1;
}

__global__ void permute_empty_kernel(const PermuteArgs a) {
  pdl_enter();
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = 0;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[e] = 0;
}

// y[t] = sum_s w ys[pos]: 2^wshift warps of a block share a token's row (one
// where there are tokens enough for every warp); KP >= k rows of NB vectors a lane
// are loaded before the first is added (in slot order).  A dropped assignment
// is a row of zeros with weight 0, so nothing of it is read.
template <typename T, int V, int KP, int NB, bool kShare>
__global__ void __launch_bounds__(kShare ? kPmThreads : kPmRowThreads)
unpermute_kernel(const UnpermuteArgs a, int wshift) {
  using P = Pack<T, V>;
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nv = a.H / V;
  if (!kShare) wshift = 0;
  const int wpt = 1 << wshift;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> (5 + wshift)) + (warp >> wshift);
  if (t >= a.T) return;
  int64_t my = lane < a.k ? a.pos[t * a.k + lane] : -1;
  if (my >= a.rows) my = -1;
  const float my_w = my < 0 ? 0.f : a.w ? a.w[t * a.k + lane] : 1.f;
  int64_t row[KP];
  float w[KP];
#pragma unroll
  for (int s = 0; s < KP; ++s) {
    row[s] = __shfl_sync(0xffffffffu, my, s);
    w[s] = __shfl_sync(0xffffffffu, my_w, s);
  }
  for (int c = (warp & (wpt - 1)) * (32 * NB) + lane; c < nv; c += 32 * NB * wpt) {
    typename P::Raw raw[KP][NB];
#pragma unroll
    for (int s = 0; s < KP; ++s)
#pragma unroll
      for (int i = 0; i < NB; ++i)
        raw[s][i] = row[s] >= 0 && c + 32 * i < nv ? row_load<T, V>(a.ys, row[s] * a.H, c + 32 * i)
                                                   : typename P::Raw{};
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (c + 32 * i >= nv) break;
      float acc[V];
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.f;
#pragma unroll
      for (int s = 0; s < KP; ++s)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(w[s], P::get(raw[s][i], j), acc[j]);
      row_store<T, V>(a.y, t * a.H, c + 32 * i, acc);
    }
  }
}

// dys[pos] = w dy, dw = <dy, ys[pos]>: dy read once, by 2^wshift warps a token
// (more than one: all the block's), whose parts of a dot product are added in
// their order.
template <typename T, int V, int KP, int NB, bool kShare>
__global__ void __launch_bounds__(kShare ? kPmThreads : kPmRowThreads)
unpermute_bwd_kernel(const UnpermuteBwdArgs a, int wshift) {
  using P = Pack<T, V>;
  pdl_enter();
  __shared__ float s_dot[kPmWarps][KP];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, nv = a.H / V;
  if (!kShare) wshift = 0;
  const int wpt = 1 << wshift;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (warps >> wshift) + (warp >> wshift);
  if (t < a.T) {
    int64_t my = lane < a.k ? a.pos[t * a.k + lane] : -1;
    if (my >= a.rows) my = -1;
    const float my_w = my >= 0 && a.w ? a.w[t * a.k + lane] : 1.f;
    int64_t row[KP];
    float w[KP], dot[KP];
#pragma unroll
    for (int s = 0; s < KP; ++s) {
      row[s] = __shfl_sync(0xffffffffu, my, s);
      w[s] = __shfl_sync(0xffffffffu, my_w, s);
      dot[s] = 0.f;
    }
    for (int c = (warp & (wpt - 1)) * (32 * NB) + lane; c < nv; c += 32 * NB * wpt) {
      typename P::Raw g[NB], raw[KP][NB];
#pragma unroll
      for (int i = 0; i < NB; ++i)
        g[i] = c + 32 * i < nv ? row_load<T, V>(a.dy, t * a.H, c + 32 * i) : typename P::Raw{};
      if (a.dw)
#pragma unroll
        for (int s = 0; s < KP; ++s)
#pragma unroll
          for (int i = 0; i < NB; ++i)
            raw[s][i] = row[s] >= 0 && c + 32 * i < nv ? row_load<T, V>(a.ys, row[s] * a.H, c + 32 * i)
                                                       : typename P::Raw{};
#pragma unroll
      for (int s = 0; s < KP; ++s) {
        if (row[s] < 0) continue;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          float v[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            if (a.dw) dot[s] = fmaf(P::get(g[i], j), P::get(raw[s][i], j), dot[s]);
            v[j] = w[s] * P::get(g[i], j);
          }
          if (c + 32 * i < nv) row_store<T, V>(a.dys, row[s] * a.H, c + 32 * i, v);
        }
      }
    }
    if (a.dw) {
      float mine = 0.f;
#pragma unroll
      for (int s = 0; s < KP; ++s) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[s] += __shfl_xor_sync(0xffffffffu, dot[s], o);
        if (lane == s) mine = dot[s];
      }
      if (kShare) {                           // the block's one token
        if (lane < KP) s_dot[warp][lane] = mine;
        __syncthreads();
        mine = 0.f;
        if (warp == 0 && lane < KP)
          for (int q = 0; q < wpt; ++q) mine += s_dot[q][lane];
      }
      if ((warp & (wpt - 1)) == 0 && lane < a.k) a.dw[t * a.k + lane] = mine;
    }
  }
  each_padding_row(a.offsets, a.counts, a.E, a.rows, static_cast<int64_t>(warp) * gridDim.x + blockIdx.x,
                   static_cast<int64_t>(gridDim.x) * warps, [&](int64_t r) {
    float zero[V];
#pragma unroll
    for (int j = 0; j < V; ++j) zero[j] = 0.f;
    for (int c = lane; c < nv; c += 32) row_store<T, V>(a.dys, r * a.H, c, zero);
  });
}

// ----------------------------------------------------------------- launches
// Blocks that own tokens: two an SM at most.
static int pm_blocks(int64_t T) {
  const int64_t most = 2 * static_cast<int64_t>(num_sms());
  return static_cast<int>(T < most ? (T > 0 ? T : 1) : most);
}
// Up to this many assignments every block counts all of them itself (T = 2048,
// k = 2: 4.6 us, of which the launch of a counting kernel would add 1.5);
// beyond, the counting kernel costs less (T = 4096, k = 2: 6.3 us against 6.8).
constexpr int64_t kPmCountOwn = 4096;

size_t permute_bytes(int64_t T, int E, int k) {
  return T * k <= kPmCountOwn ? 0 : 4 * static_cast<size_t>(E) * pm_blocks(T);
}

bool permute_counts_first(int64_t T, int k) { return T * k > kPmCountOwn; }

// Writes bound the copy (this GPU fills memory at 3.7-4.0 TB/s, against 6.8 of
// a copy's two directions together).  From 256 MB of rows on, the tables are
// made alone and the rows copied by the gradient's kernel, whose small blocks
// even out the SMs' paces: T = 16384, k = 4, H = 4096 (537 MB) 128 -> 119 us;
// at T = 16384, k = 2, H = 2048 (134 MB) the launch costs what it gives.
static bool pm_copy_apart(int64_t T, int k, int row_bytes) { return T * k * row_bytes >= (256ll << 20); }

static int pm_tokens(const PermuteArgs& a) {
  const int b = pm_blocks(a.T);
  return static_cast<int>((a.T + b - 1) / b);
}
// The blocks that do own a token (the last of pm_blocks may be left without).
static int pm_owners(const PermuteArgs& a) { return static_cast<int>((a.T + pm_tokens(a) - 1) / pm_tokens(a)); }

cudaError_t launch_permute_count(const PermuteArgs& a, cudaStream_t st) {
  return launch_dependent_kernel(permute_count_kernel, dim3(pm_owners(a)), dim3(128), 0, st, a, pm_tokens(a),
                                 static_cast<int32_t*>(a.scratch));
}

cudaError_t launch_permute(int dtype, const PermuteArgs& a, cudaStream_t st) {
  if (a.T == 0) return launch_dependent_kernel(permute_empty_kernel, dim3(1), dim3(128), 0, st, a);
  const int row_bytes = a.H * (dtype == kDtypeBF16 ? 2 : 4);
  const int32_t* cnt = permute_counts_first(a.T, a.k) ? static_cast<const int32_t*>(a.scratch) : nullptr;
  // and blocks for the padding, where the tokens' own would take long over it
  const int owners = pm_owners(a);
  const int64_t pad = (a.rows - a.T * a.k + 3) / 4, most = pm_blocks(int64_t{1} << 40);
  const int grid = static_cast<int>(pad < owners ? owners : pad < most ? pad : most);
  auto run = [&](auto kern) {
    return launch_dependent_kernel(kern, dim3(grid > owners ? grid : owners), dim3(kPmThreads), 0, st, a, pm_tokens(a),
                                   owners, cnt, row_bytes, pm_copy_apart(a.T, a.k, row_bytes) ? 0 : 1);
  };
  if (row_bytes % 16 == 0) return run(permute_kernel<uint4>);
  if (row_bytes % 8 == 0) return run(permute_kernel<uint2>);
  if (row_bytes % 4 == 0) return run(permute_kernel<uint32_t>);
  return run(permute_kernel<uint16_t>);
}

static inline int pm_kp(int k) { return k <= 1 ? 1 : k <= 2 ? 2 : k <= 4 ? 4 : 8; }
// Warps that share a token: one, and more where there are fewer tokens than
// eight warps an SM, as far as the row has pieces of `piece` vectors for them
// (T = 4, k = 7, H = 7424, bf16: 17.6 us with one warp a token).
// log2 of it.
static int pm_wshift(int64_t T, int nv, int piece) {
  int s = 0;
  while ((1 << s) < kPmWarps && (T << s) < 8ll * num_sms() && (piece << s) < nv) ++s;
  return s;
}
// Blocks of 128 threads, or of one token's warps; `more` rows of padding may
// want more of them.
static void pm_row_grid(int64_t T, int wshift, int64_t more, dim3& grid, dim3& block) {
  const int wpt = 1 << wshift;
  const int warps = wpt > 1 ? wpt : kPmRowThreads / 32;
  const int64_t own = wpt > 1 ? T : (T + warps - 1) / warps;
  const int64_t pad = (more + 1) / 2, most = 4 * static_cast<int64_t>(num_sms());
  const int64_t want = pad < most ? pad : most;
  grid = dim3(static_cast<unsigned>(own > want ? own : want));
  block = dim3(32 * warps);
}

// Narrow accesses (rows that are not 16-byte aligned): more of them in flight.
template <typename T, int V>
constexpr int pm_wide() { return V * sizeof(T) == 16 ? 1 : V * sizeof(T) == 8 ? 2 : 4; }

template <typename T, int V, int KP, int NB>
static cudaError_t unpermute_run(const UnpermuteArgs& a, cudaStream_t st) {
  const int wshift = pm_wshift(a.T, a.H / V, 32 * NB);
  dim3 grid, block;
  pm_row_grid(a.T, wshift, 0, grid, block);
  auto kern = wshift > 0 ? unpermute_kernel<T, V, KP, NB, true> : unpermute_kernel<T, V, KP, NB, false>;
  return launch_dependent_kernel(kern, grid, block, 0, st, a, wshift);
}
template <typename T, int V>
static cudaError_t unpermute_pick(const UnpermuteArgs& a, cudaStream_t st) {
  constexpr int kWide = pm_wide<T, V>();
  switch (pm_kp(a.k)) {
    case 1: return unpermute_run<T, V, 1, 4 * kWide>(a, st);
    case 2: return unpermute_run<T, V, 2, 4 * kWide>(a, st);
    case 4: return unpermute_run<T, V, 4, 2 * kWide>(a, st);
    default: return unpermute_run<T, V, 8, kWide>(a, st);
  }
}
cudaError_t launch_unpermute(int dtype, const UnpermuteArgs& a, cudaStream_t st) {
  if (dtype == kDtypeBF16) {
    if (a.H % 8 == 0) return unpermute_pick<__nv_bfloat16, 8>(a, st);
    if (a.H % 4 == 0) return unpermute_pick<__nv_bfloat16, 4>(a, st);
    if (a.H % 2 == 0) return unpermute_pick<__nv_bfloat16, 2>(a, st);
    return unpermute_pick<__nv_bfloat16, 1>(a, st);
  }
  if (a.H % 4 == 0) return unpermute_pick<float, 4>(a, st);
  if (a.H % 2 == 0) return unpermute_pick<float, 2>(a, st);
  return unpermute_pick<float, 1>(a, st);
}

template <typename T, int V, int KP>
static cudaError_t unpermute_bwd_run(const UnpermuteBwdArgs& a, cudaStream_t st) {
  constexpr int kWide = pm_wide<T, V>();
  const int wshift = pm_wshift(a.T, a.H / V, 32 * kWide);
  dim3 grid, block;
  pm_row_grid(a.T, wshift, a.rows > a.T * a.k ? a.rows - a.T * a.k : 0, grid, block);
  auto kern = wshift > 0 ? unpermute_bwd_kernel<T, V, KP, kWide, true> : unpermute_bwd_kernel<T, V, KP, kWide, false>;
  return launch_dependent_kernel(kern, grid, block, 0, st, a, wshift);
}
template <typename T, int V>
static cudaError_t unpermute_bwd_pick(const UnpermuteBwdArgs& a, cudaStream_t st) {
  switch (pm_kp(a.k)) {
    case 1: return unpermute_bwd_run<T, V, 1>(a, st);
    case 2: return unpermute_bwd_run<T, V, 2>(a, st);
    case 4: return unpermute_bwd_run<T, V, 4>(a, st);
    default: return unpermute_bwd_run<T, V, 8>(a, st);
  }
}
cudaError_t launch_unpermute_bwd(int dtype, const UnpermuteBwdArgs& a, cudaStream_t st) {
  if (dtype == kDtypeBF16) {
    if (a.H % 8 == 0) return unpermute_bwd_pick<__nv_bfloat16, 8>(a, st);
    if (a.H % 4 == 0) return unpermute_bwd_pick<__nv_bfloat16, 4>(a, st);
    if (a.H % 2 == 0) return unpermute_bwd_pick<__nv_bfloat16, 2>(a, st);
    return unpermute_bwd_pick<__nv_bfloat16, 1>(a, st);
  }
  if (a.H % 4 == 0) return unpermute_bwd_pick<float, 4>(a, st);
  if (a.H % 2 == 0) return unpermute_bwd_pick<float, 2>(a, st);
  return unpermute_bwd_pick<float, 1>(a, st);
}

bool permute_copies_apart(int dtype, const PermuteArgs& a) {
  return pm_copy_apart(a.T, a.k, a.H * (dtype == kDtypeBF16 ? 2 : 4));
}
cudaError_t launch_permute_rows(int dtype, const PermuteArgs& a, cudaStream_t st) {
  return launch_unpermute_bwd(dtype, UnpermuteBwdArgs{a.x, nullptr, a.pos, nullptr, a.offsets, a.counts, a.xs, nullptr,
                                                      a.T, a.rows, a.H, a.E, a.k}, st);
}

}  // namespace mm

// tt_gemm.cuh - matrix products of 16-bit operands on the tensor cores, with an
// epilogue of the caller's: D = A * B^T in 32 bits, tile by tile.
//
// A pair of SMs computes a tile of 256 x 256: each loads half of A's rows and half
// of B's by TMA (64 of the contraction a stage), one thread of the pair issues the
// products (tcgen05, cta_group::2), and 128 rows of the result lie in the tensor
// memory of each.  Two tiles fit there, so that the epilogue's warps read one while
// the next is computed.  A launch has a pair for every two SMs; tiles are handed out
// by number.
//
// An operand lies in memory either with the contraction along its rows ("K-major")
// or across them ("MN-major"); both are what a TMA box of 64 elements by 8 rows and
// more leaves in shared memory with the 128-byte swizzle.  An operand may be a sum
// of up to three parts (32-bit values split into bfloat16 ones): then the products
// of the listed pairs of parts are added up.
//
// 64 of the contraction of a tile take 0.31 us at the clocks that the power limit leaves
// (0.27 at the highest), a tile 0.45 us more.  The tensor pipe is active for 88% of the cycles
// with a contraction of 2048 and 96% with one of 25,000; without its epilogue's work the
// loss of 4096 x 100256 takes as long (862 us and 861).  Five stages instead of six are as
// fast, and tile rows passed through by 8 or 4 instead of 16 take 2 and 4% longer.
// Clusters of two pairs, with B's halves multicast, would leave 8 SMs idle, which they do not
// fit.
#pragma once
#include <cuda.h>

#include "tt_ops.cuh"
#include "tt_plan.h"

namespace tt {
namespace gemm {

using namespace tt::ops;

constexpr int STAGES = 6, STAGE_BYTES = 2 * HALF * KB * 2;
constexpr int EPI_WARPS = 8, THREADS = (4 + EPI_WARPS) * 32;
constexpr int OWN_BYTES = 4096;                            // shared memory of an epilogue's warp, for what it writes
constexpr int SHARED = STAGES * STAGE_BYTES + EPI_WARPS * OWN_BYTES + 1024;   // and what aligns the stages to 1024 bytes

struct Gemm {
  int m_tiles, n_tiles, splits;                           // the contraction is cut into `splits` parts
  int k_blocks;                                           // of 64, the last filled up with zeros
  int rows_a, rows_b;                                     // of the operands
  uint32_t box_a;                                         // bytes of A a block loads a stage
  int pairs;                                              // of parts, listed in nibbles of pair_a and pair_b
  uint32_t pair_a, pair_b, idesc;
  int group;                                              // tile rows that are passed through together
  const int32_t *only;                                    // or NULL: nothing is done unless only[0], for the tile rows i with only[1 + i]
  int32_t *status;
};

// ------------------------------------------------------------ device: waits
__device__ __forceinline__ uint32_t saddr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t in_block(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok;
}
// false: the wait ran out, here or in another role of the block
__device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile int *dead) {
  uint64_t now;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
  Patience patience(now);
  for (uint32_t i = 0; i < 1u << 30; ++i) {
    if (bar_try(bar, parity)) return true;
    if ((i & 63) == 63) {
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
      if (*dead || patience.over(now)) break;
    }
  }
  *dead = 1;
  return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *dead) {
  return bar_try(bar, parity) || bar_wait_long(bar, parity, dead);
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// a barrier of another block, told that tensor memory has been read: nothing else is
// ordered by it (a release at cluster scope waits for the warp's stores)
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------------------ device: copies and products
// a box to this block's shared memory, its bytes told to a barrier of the pair
__device__ __forceinline__ void load_box(uint32_t to, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::
                   "r"(to), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
               "l"(b), "r"(idesc), "r"((uint32_t)add)
               : "memory");
}
// the barrier at this address of both blocks, when the products issued so far are done
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"((uint16_t)3)
               : "memory");
}
// 32 columns of a warp's rows; they are there behind tmem_wait, which has to be given them
__device__ __forceinline__ void tmem_load32(uint32_t at, float v[32]) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_wait(float v[64]) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]), "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]), "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]), "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
               :
               : "memory");
}

// A shared memory descriptor: the address and two distances in units of 16 bytes,
// version 1, 128-byte swizzle.  K-major: groups of eight rows (of 128 bytes) lie
// `stride` apart.  MN-major: eight of the contraction lie `stride` apart, 64 of the
// rows `lead`.
__device__ __forceinline__ uint64_t smem_desc(uint32_t at, uint32_t lead, uint32_t stride) {
  return (uint64_t)((at & 0x3FFFF) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// 16 bytes of the warp's own shared memory: 32 rows of 128 bytes, swizzled as TMA's
// 128-byte mode does, so that rows can be written and columns of chunks be read
__device__ __forceinline__ uint32_t own_chunk(uint32_t own, int row, int chunk) { return own + row * 128 + ((chunk ^ (row & 7)) << 4); }
__device__ __forceinline__ void own_write(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 own_read(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float own_float(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
// 32 rows of 64 16-bit elements from there to a matrix, by one thread; what lies outside is left out
__device__ __forceinline__ void store_box(const CUtensorMap *map, int x, int y, int z, uint32_t own) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map), "r"(own), "r"(x), "r"(y),
               "r"(z)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void fence_copies() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// how a block's half of an operand (128 rows by 64 of the contraction) is loaded
// and described: K-major one box of 128 rows, MN-major two boxes of 64 rows
template <bool MN> struct Operand {
  static __device__ __forceinline__ void load(uint32_t to, const CUtensorMap *map, int row, int k, int part, uint32_t bar) {
    if (MN) {
      load_box(to, map, row, k, part, bar);
      load_box(to + HALF * KB, map, row + 64, k, part, bar);
    } else {
      load_box(to, map, k, row, part, bar);
    }
  }
  // of the 16 of the contraction from 16 * step on
  static __device__ __forceinline__ uint64_t desc(uint32_t at, int step) {
    return MN ? smem_desc(at + step * 2048, HALF * KB, 1024) : smem_desc(at + step * 32, 16, 1024);
  }
};

// tile number -> its place: `group` tile rows are passed through together, column by
// column, so that what runs at a time shares operands of both sides
struct Place {
  int t, m, n, split;                                     // t: the tile's number, n_tiles for none
  int first, last;                                        // blocks of the contraction
};
// The next tile of a pair of SMs at or behind number t.  The threads that copy and multiply
// ask for it when they are done with one: within their loops it slows every step (4096 x
// 100256 x 2048 scored: 845 us, and 875).
__device__ __forceinline__ Place place_of(const Gemm &g, int t, int n_tiles, int step) {
  Place p;
  p.split = p.first = 0;
  p.last = g.k_blocks;
  for (;; t += step) {
    p.t = min(t, n_tiles);
    if (t >= n_tiles) break;
    int i = t;
    const int per = g.m_tiles * g.n_tiles;
    if (g.splits > 1) {
      p.split = i / per;
      i -= p.split * per;
      p.first = (uint32_t)(g.k_blocks * p.split) / (uint32_t)g.splits;
      p.last = (uint32_t)(g.k_blocks * (p.split + 1)) / (uint32_t)g.splits;
    }
    const int first = i / (g.group * g.n_tiles) * g.group, rows = min(g.group, g.m_tiles - first);
    i -= first * g.n_tiles;
    p.n = i / rows;
    p.m = first + i - p.n * rows;
    if (!g.only || g.only[1 + p.m]) break;
  }
  return p;
}

// Epi is called by the epilogue's warps as epi(row, column, split, own, begun, load, release): the
// row of the result that a thread has (consecutive ones in a warp), the first of the 128
// columns that it reads, the warp's own shared memory, what epi.begin(row) gave before the tile was there, load(c, v), which brings 64 of the
// columns from the c-th on, and release(), which follows the last of them: the next
// products may overwrite them.  Both are called by whole warps.  epi.end() comes behind
// the last tile.
template <bool A_MN, bool B_MN, class Epi>
__global__ void __cluster_dims__(2) __launch_bounds__(THREADS, 1)
    k_gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const Gemm g,
           const __grid_constant__ Epi epi) {
  let_next_start();
  if (g.only) {
    wait_for_last();
    if (!g.only[0]) return;
  }
  extern __shared__ uint8_t s_raw[];
  __shared__ uint64_t s_bar[2 * STAGES + 4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const uint32_t stages = (saddr(s_raw) + 1023) & ~1023u;
  const uint32_t full = saddr(s_bar), empty = full + 8 * STAGES, done = empty + 8 * STAGES, free_ = done + 16;
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(done + 8 * i, 1);
      bar_init(free_ + 8 * i, 2 * EPI_WARPS);
    }
    s_dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *(volatile uint32_t *)&s_tmem;
  wait_for_last();                                        // all else is a matter of this block
  const int n_tiles = g.m_tiles * g.n_tiles * g.splits, n_pairs = gridDim.x / 2;
  bool ok = true;

  if (warp == 0 && lane == 0) {
    // copies: a stage is free when the products that read it are done
    int stage = 0;
    uint32_t phase = 1;
    for (Place p = place_of(g, blockIdx.x / 2, n_tiles, n_pairs), next; ok && p.t < n_tiles; p = next) {
      const int ra = p.m * TILE + rank * HALF, rb = p.n * TILE + rank * HALF;
      // Rows that are not there are left out: what lies in their place enters only results
      // of theirs.  (TMA reads the border again for each row beyond it: 152 SMs at one
      // line of a single row took 124 us for 1 x 100256 x 2048 instead of 86.)
      const uint32_t bytes = (1 + (p.m * TILE + HALF < g.rows_a)) * g.box_a + (1 + (p.n * TILE + HALF < g.rows_b)) * (STAGE_BYTES / 2);
      auto copy = [&](int i, int k) {
        if (!(ok = bar_wait(empty + 8 * stage, phase, &s_dead))) return false;
        if (rank == 0) bar_expect(full + 8 * stage, bytes);
        const uint32_t bar = in_block(full + 8 * stage, 0), to = stages + stage * STAGE_BYTES;
        if (ra < g.rows_a) Operand<A_MN>::load(to, &map_a, ra, k * KB, g.pair_a >> (4 * i) & 15, bar);
        if (rb < g.rows_b) Operand<B_MN>::load(to + STAGE_BYTES / 2, &map_b, rb, k * KB, g.pair_b >> (4 * i) & 15, bar);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
        return true;
      };
      if (g.pairs == 2 || g.pairs == 3) {
        // all of a block of the contraction: its second reading comes from L2
        for (int k = p.first; ok && k < p.last; ++k)
          for (int i = 0; i < g.pairs; ++i)
            if (!copy(i, k)) break;
      } else {
        for (int i = 0; ok && i < g.pairs; ++i)
          for (int k = p.first; k < p.last; ++k)
            if (!copy(i, k)) break;
      }
      next = place_of(g, p.t + n_pairs, n_tiles, n_pairs);
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    int stage = 0;
    uint32_t phase = 0;
    int i = 0;
    for (Place p = place_of(g, blockIdx.x / 2, n_tiles, n_pairs), next; ok && p.t < n_tiles; p = next) {
      const int count = (p.last - p.first) * g.pairs;
      if (!(ok = bar_wait(free_ + 8 * (i & 1), (i >> 1 & 1) ^ 1, &s_dead))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = tmem + (i & 1) * TILE;
      for (int k = 0; k < count; ++k) {
        if (!(ok = bar_wait(full + 8 * stage, phase, &s_dead))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t at = stages + stage * STAGE_BYTES;
#pragma unroll
        for (int s = 0; s < KB / 16; ++s)
          mma(d, Operand<A_MN>::desc(at, s), Operand<B_MN>::desc(at + STAGE_BYTES / 2, s), g.idesc, k || s);
        commit(empty + 8 * stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (ok) commit(done + 8 * (i & 1));
      ++i;
      next = place_of(g, p.t + n_pairs, n_tiles, n_pairs);
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    int i = 0;
    const uint32_t own = stages + STAGES * STAGE_BYTES + (warp - 4) * OWN_BYTES;
    for (Place p = place_of(g, blockIdx.x / 2, n_tiles, n_pairs), next; p.t < n_tiles; p = next) {
      next = place_of(g, p.t + n_pairs, n_tiles, n_pairs);
      const int row = p.m * TILE + (int)rank * HALF + quarter * 32 + lane;
      const auto begun = epi.begin(row);
      ok = bar_wait(done + 8 * (i & 1), i >> 1 & 1, &s_dead);
      if (!__all_sync(~0u, ok)) {
        ok = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t at = tmem + (i & 1) * TILE + half * HALF + ((uint32_t)(quarter * 32) << 16);
      epi(row, p.n * TILE + half * HALF, p.split, own, begun,
          [&](int c, float v[64]) {
            tmem_load32(at + c, v);
            tmem_load32(at + c + 32, v + 32);
            tmem_wait(v);
          },
          [&]() {
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) bar_arrive_cluster(in_block(free_ + 8 * (i & 1), 0));
          });
      ++i;
    }
    epi.end();
  }
  if (!ok) {
    // what is under way (copies, products) ends by itself within this time
    op_status(g.status, TT_ERR_TIMEOUT);
    for (int i = 0; i < 2000; ++i) __nanosleep(1000);
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  if (warp == 2) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ------------------------------------------------------------ host
// A matrix of up to three parts in 16-bit elements, 16-byte aligned: what a TMA map needs.
struct Matrix {
  const void *p;
  int64_t rows, cols, stride, parts, part_stride;          // in elements
};

CUresult encode_map(CUtensorMap *map, bool bf16, const Matrix &m, uint32_t box_rows);

inline uint32_t idesc_of(bool bf16, bool a_mn, bool b_mn) {
  const uint32_t type = bf16 ? 1 : 0;
  return 1u << 4 | type << 7 | type << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (TILE >> 3) << 17 | (TILE >> 4) << 24;
}

template <bool A_MN, bool B_MN, class Epi> struct GemmTag {};

// All launches of a call are chained, the first one to whatever the caller's stream has
// before it: a kernel's blocks start, and set themselves up, while the one before ends, and
// wait for all of it before they read or write memory.
// D [rows of a][rows of b] = a * b^T over the contraction; with _MN the matrix lies the
// other way round (its rows are the contraction).  False: an error, which is kept, or more
// parts of the contraction than it has blocks.
template <bool A_MN, bool B_MN, class Epi>
inline bool run_gemm(bool bf16, const Matrix &a, const Matrix &b, int splits, int group, const Epi &epi, int32_t *status,
                     cudaStream_t stream, const int32_t *only = nullptr) {
  CUtensorMap ma, mb;
  // few rows: a box no higher than they are
  const int64_t rows_a = A_MN ? a.cols : a.rows, rows_b = B_MN ? b.cols : b.rows;
  const uint32_t box = A_MN ? HALF : (uint32_t)std::min<int64_t>(HALF, (rows_a + 7) / 8 * 8);
  if (encode_map(&ma, bf16, a, A_MN ? KB : box) != CUDA_SUCCESS || encode_map(&mb, bf16, b, B_MN ? KB : HALF) != CUDA_SUCCESS) return false;
  Gemm g;
  g.rows_a = (int)rows_a;
  g.rows_b = (int)rows_b;
  g.box_a = box * KB * 2;
  g.m_tiles = (int)((rows_a + TILE - 1) / TILE);
  g.n_tiles = (int)((rows_b + TILE - 1) / TILE);
  g.k_blocks = (int)(((A_MN ? a.rows : a.cols) + KB - 1) / KB);
  if (splits > g.k_blocks) return false;
  g.splits = splits;
  // The products of parts whose orders add up to less than three (two parts: two), the
  // smallest first (the sums are cut off, not rounded, at each step: small ones lose less).
  // Three parts each: (2,0) (0,2) (1,1) (1,0) (0,1) (0,0), the rest is below 2^-24; two and
  // two: (1,0) (0,1) (0,0); two and one: (1,0) (0,0); one and two: (0,1) (0,0).
  g.pairs = pairs_of((int)a.parts, (int)b.parts);
  g.pair_a = g.pairs == 6 ? 0x001102 : a.parts == 2 ? 0x001 : 0;
  g.pair_b = g.pairs == 6 ? 0x010120 : g.pairs == 3 ? 0x010 : b.parts == 2 ? 0x001 : 0;
  g.idesc = idesc_of(bf16, A_MN, B_MN);
  g.group = group;
  g.only = only;
  g.status = status;
  auto k = k_gemm<A_MN, B_MN, Epi>;
  if (allow_shared<GemmTag<A_MN, B_MN, Epi>>(k, SHARED)) return false;
  const int tiles = g.m_tiles * g.n_tiles * g.splits;
  launch_cluster(k, dim3(2 * std::min(tiles, SMS / 2)), THREADS, SHARED, 1, true, stream, ma, mb, g, epi);
  return true;
}

}  // namespace gemm
}  // namespace tt

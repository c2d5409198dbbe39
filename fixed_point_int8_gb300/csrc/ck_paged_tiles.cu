// Attention of chunks of new tokens over a cache in pages, on the tensor cores ("Attention,
// stage by stage"): 128 queries (rows x heads that share a key head) of one sequence at a time.
//
// Exactness.  Queries, keys and values that fit three balanced digits of 8 bits (x = d0 + 2^8 d1
// + 2^16 d2, every d in -128 .. 127: |x| up to 127.5 with 16 fraction bits) are split into f16
// planes, so a product is nine products of planes.  Products of digits are exact, and an f32
// accumulator is exact while the sum of the magnitudes stays below 2^24:
//   scores: products of equal weight share an accumulator, at most three pairs over at most 128
//     elements: 3 * 128 * 2^14 < 2^23;
//   values: a probability P (24 fraction bits) has the unsigned digits p0, p1, p2, and the P of
//     a row add up to at most 2^24, so sum p1 <= 2^16 and sum p2 <= 2^8.  Over 256 positions the
//     accumulator of weight 2^0 stays below 255 * 128 * 256, that of 2^8 below twice that (just
//     under 2^24), that of 2^16 at most 255 * 128 * 256 + 128 * 2^16 + 2^15 = 2^24, which f32 holds
//     (and is below: the P add up to 2^24, so sum p1 <= 2^16 - 255 where sum p0 = 255 * 256), and
//     those of 2^24 and 2^32 together, in units of 2^24, below 2^23 + 2^15: they share one.  The
//     planes carry powers of two (2^-12, 2^-4, 2^4) so that the products come out aligned.
//     After 256 positions the four accumulators move into 64-bit integers.
// The exponential depends on the row's maximum and the probability on its sum, and both are
// floored table and quotient values that cannot be rescaled: scores go to a scratch as 32-bit
// words (a score that does not fit, and any digit that does not, hands the tile to the kernel
// for all values), then maximum, sum and weighted values follow in three passes.
//
// The instructions around the products bound it (about 70 a score, a third of the issue slots in
// phases that wait for one another), and the scratch's traffic where it is larger than L2: 256 rows
// over 7,936 positions of 32 heads of 64 take 358 us, chunks of 201 and 151 rows over 2,047 and 777
// of 32 heads of 128 take 251.  Twice the warps with 64 registers a thread were slower (447 against
// 388 us, 276 against 255 then), and so were 16-bit places in the table in the scratch for the
// exponentials (346 against 338, 243 against 234 then).  A thread owns a row (its lane of tensor
// memory), so maxima and sums need no exchange inside a warp.  A cluster splits a tile's positions,
// which fills the GPU when tiles are few; it exchanges maxima, sums and the 64-bit sums of values
// through distributed shared memory.
#include "ck_paged_attention.cuh"
#include "ck_tc.cuh"

namespace ck {
namespace {

constexpr uint32_t kTileRows = 128, kTilePos = 32, kBlockPos = 64, kFlushBlocks = 4;
constexpr uint32_t kDiags = 5;
// scores on their way back: four stages of 32 positions, [position / 4][row][4] as in the scratch
constexpr uint32_t kRing = 4, kStage = kTilePos * kTileRows * 4;

template <int HD>
struct Tile {
  // groups of 128 threads, in each a thread a row
  static constexpr uint32_t kThreads = 4 * HD, kGroups = HD / 32;
  static constexpr uint32_t kBufs = HD == 64 ? 1 : 2;              // score accumulators, operand buffers
  static constexpr uint32_t kTmem = HD == 64 ? 256 : 512;          // two blocks an SM for head size 64
  static constexpr uint32_t kScoreCol = 3 * HD / 2;                // behind the query digits
  // [64 elements][place][position]: two buffers of three key planes, two places of zeros around each
  static constexpr uint32_t kKeyPlane = kTilePos * 128, kKeyHalf = 12 * kKeyPlane, kKeys = (HD / 64) * kKeyHalf;
  static constexpr uint32_t kProbPlane = kTileRows * 128, kValuePlane = HD * 128;
  static constexpr uint32_t kValueBuf = 3 * (kProbPlane + kValuePlane);
  static constexpr uint32_t kPitch = kTileRows + 1;  // of the 64-bit sums, [element][row]
  static constexpr uint32_t max3(uint32_t a, uint32_t b, uint32_t c) {
    return a > b ? (a > c ? a : c) : (b > c ? b : c);
  }
  static constexpr uint32_t kTurn = (kThreads / 32) * 48 * 33 * 4;  // query digits on their way to tensor memory
  static constexpr uint32_t kOperands =
      (max3(kKeys, kBufs * kValueBuf, max3(HD * kPitch * 8, kTurn, 0)) + 1023) & ~1023u;
  static constexpr uint32_t kTableOff = kOperands, kTableBytes = 4097 * 4 + 12;
  static constexpr uint32_t kRedOff = kTableOff + kTableBytes;   // [groups][128] u64
  static constexpr uint32_t kMaxOff = kRedOff + kGroups * kTileRows * 8;  // [128] i32
  static constexpr uint32_t kSumOff = kMaxOff + kTileRows * 4;   // [128] u64
  static constexpr uint32_t kMiscOff = kSumOff + kTileRows * 8;  // barrier, tensor memory, flags
  static constexpr uint32_t kRingOff = kMiscOff + 64;            // the scores' barriers
  static constexpr uint32_t kSmem = kRingOff + kRing * 16 + 1024; // + alignment of the operands
  static_assert(kRing * kStage <= kOperands, "the scores' ring");
  static_assert(kScoreCol + kBufs * kDiags * kTilePos <= kTmem && 4 * HD <= kTmem, "tensor memory");
};

__device__ __forceinline__ uint32_t tile_idesc(uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | ((kTileRows >> 4) << 24); }

// One product, issued by the warp's elected lane: the whole warp computes the operands, so that
// they stay in uniform registers (a branch of one lane would move each there by itself, which
// measured 68 cycles a product against about 20).
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }"
      ::"r"(smem_addr(bar)), "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elected() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_operands() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(addr));
}
// The words are there after the wait; the second statement reads and writes each of them, so that
// the compiler moves nothing that uses them before it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[N][8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile("" : "+r"(v[i][0]), "+r"(v[i][1]), "+r"(v[i][2]), "+r"(v[i][3]), "+r"(v[i][4]), "+r"(v[i][5]),
                      "+r"(v[i][6]), "+r"(v[i][7]));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Balanced digits: the bytes of x + 0x808080 are the digits plus 128, when x fits them.
__device__ __forceinline__ uint32_t biased(int32_t x) { return (uint32_t)x + 0x808080u; }
// Two digit bytes at nibble selectors of w as f16: 0x64BB is 1024 + BB exactly.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t lift(uint32_t w) {
  return __byte_perm(w, 0x64646464u, SEL);
}
__device__ __forceinline__ uint32_t sub_1152(uint32_t h) {  // balanced digits, unscaled
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
  return r;
}
__device__ __forceinline__ uint32_t fma_h2(uint32_t h, uint32_t scale, uint32_t bias) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(h), "r"(scale), "r"(bias));
  return r;
}
// f16 pairs of the plane scales 2^-12, 2^-4, 2^4 and of the offsets they take away:
// 1152 * scale for balanced digits, 1024 * scale for unsigned ones (all exact).
constexpr uint32_t kScale0 = 0x0C000C00u, kScale1 = 0x2C002C00u, kScale2 = 0x4C004C00u;
constexpr uint32_t kBal0 = 0xB480B480u, kBal1 = 0xD480D480u, kBal2 = 0xF480F480u;   // -0.28125, -72, -18432
constexpr uint32_t kUns0 = 0xB400B400u, kUns1 = 0xD400D400u, kUns2 = 0xF400F400u;   // -0.25, -64, -16384

__device__ __forceinline__ uint32_t peer32(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long peer64(const void* p, uint32_t rank) {
  uint32_t a;
  unsigned long long v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void all_sync(uint32_t C) {  // the cluster's threads, or the block's
  if (C > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
}

template <int HD>
__global__ void __launch_bounds__(Tile<HD>::kThreads, HD == 64 ? 2 : 1) k_pattn_tiles(const TilesParams f) {
  using T = Tile<HD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const PAttnParams& p = f.a;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cg = warp >> 2, r = 32 * (warp & 3) + lane;  // column group and row of this thread
  const uint32_t lane_base = (32 * (warp & 3)) << 16;
  uint32_t C, rank, clusters, cluster;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%nclusterid.x;" : "=r"(clusters));
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(cluster));
  uint32_t* table_s = reinterpret_cast<uint32_t*>(sm + T::kTableOff);
  unsigned long long* red = reinterpret_cast<unsigned long long*>(sm + T::kRedOff);
  int32_t* xmax = reinterpret_cast<int32_t*>(sm + T::kMaxOff);
  unsigned long long* xsum = reinterpret_cast<unsigned long long*>(sm + T::kSumOff);
  // Barriers, two of a kind used in turn: operands of a batch of products in place (and the
  // accumulators free), the products done, a tile's accumulators drained.
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + T::kMiscOff);
  uint64_t* done = full + 2;
  uint64_t* drained = full + 4;
  uint64_t* ring = reinterpret_cast<uint64_t*>(sm + T::kRingOff);  // a stage of scores has come
  uint64_t* freed = ring + kRing;                                   // and has been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + T::kMiscOff + 48);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + T::kMiscOff + 52);
  uint32_t* next_s = reinterpret_cast<uint32_t*>(sm + T::kMiscOff + 60);
  uint32_t* bad_s = reinterpret_cast<uint32_t*>(sm + T::kMiscOff + 56);  // this block's reason to give the tile away

  for (uint32_t i = tid; i < 4097; i += T::kThreads) table_s[i] = min(__ldg(p.exp_tab + i), 1u << 30);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mb_init(full + i, T::kThreads / 32);
      mb_init(done + i, 1);
      mb_init(drained + i, T::kThreads / 32);
    }
    for (uint32_t i = 0; i < kRing; ++i) {
      mb_init(ring + i, 1);
      mb_init(freed + i, T::kThreads / 32);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(tmem_slot)), "r"(T::kTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot, tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
  const uint32_t warp_u = __shfl_sync(0xffffffffu, warp, 0);  // known to be the same in the warp
  const uint64_t operands = smem_desc(smem_addr(sm));
  constexpr uint32_t kWarps = T::kThreads / 32;
  uint32_t batch = 0, tiles = 0, staged = 0;  // batches, tiles and stages so far: the barriers' phases
  auto wait_full = [&](uint32_t g) { mb_wait(full + (g & 1u), (g >> 1) & 1u, const_cast<volatile int*>(abort_flag)); tc_after(); };
  auto wait_done = [&](uint32_t g) { mb_wait(done + (g & 1u), (g >> 1) & 1u, const_cast<volatile int*>(abort_flag)); tc_after(); };
  auto wait_drained = [&](uint32_t g) { mb_wait(drained + (g & 1u), (g >> 1) & 1u, const_cast<volatile int*>(abort_flag)); tc_after(); };
  auto wait_copy = [&](uint64_t* b, uint32_t parity) {  // also when giving up: no block ends before its copies
    for (uint32_t it = 0; it < kTcPoll; ++it)
      if (mb_try(b, parity)) return;
    *abort_flag = 1;
  };
  auto arrive = [&](uint64_t* b) {  // this warp's accesses so far come before the phase
    tc_before();
    __syncwarp();
    if (lane == 0) mb_arrive(b);
  };

  const uint32_t shift = p.pool.page_shift, pmask = (1u << shift) - 1;
  const uint32_t group = p.heads / p.pool.kv_heads;
  // [position / 4][row][4]: a thread writes and reads four positions of its row at once
  int4* scores = reinterpret_cast<int4*>(f.scores) + (size_t)blockIdx.x * (f.cap / 4) * kTileRows;
  // [element][thread]: the 64-bit sums between flushes
  unsigned long long* kept = f.sums + (size_t)blockIdx.x * 32 * T::kThreads + tid;
  const uint64_t per_seq = (uint64_t)p.pool.kv_heads * f.tiles;
  const uint64_t items = (uint64_t)p.batch.seqs * per_seq;

  // a cluster's first tile is its number's, the next ones come from a count that all draw from
  uint64_t item = cluster;
  while (item < items) {
    const uint32_t seq = (uint32_t)(item / per_seq), rest = (uint32_t)(item - seq * per_seq);
    const uint32_t kvh = rest / f.tiles, v0 = (rest - kvh * f.tiles) * kTileRows;
    const Sequence sq = load_sequence(p.batch, seq, shift);
    if (!sq.ok) {
      if (tid == 0 && rank == 0) note(p.batch, seq, err_key(0, p.pool.layer, CK_PAGED_BAD_SEQUENCE, 0));
    }
    const uint32_t queries = sq.ok ? sq.count * group : 0;
    if (tid == 0 && rank == 0) *next_s = clusters + atomicAdd(f.any + 1, 1u);
    if (v0 >= queries) {  // (for every block of the cluster)
      all_sync(C);
      const uint32_t then = C > 1 ? peer32(next_s, 0) : *next_s;
      all_sync(C);
      item = then;
      continue;
    }
    const uint32_t v = v0 + r, last = min(queries, v0 + kTileRows) - 1;
    auto seen_by = [&](uint32_t q) {  // positions query q sees
      const uint32_t up = q / group + sq.len;
      return up >= sq.count ? up - sq.count + 1 : 0;
    };
    const uint32_t top = seen_by(last), np = v < queries ? seen_by(v) : 0;
    const uint32_t per = ((top + C - 1) / C + kBlockPos - 1) & ~(kBlockPos - 1);
    const uint32_t c0 = min(top, rank * per), n = min(top, c0 + per) - c0;
    const uint32_t lim = np > c0 ? min(n, np - c0) : 0;  // positions of this block that the row sees
    const uint32_t nt = (n + kTilePos - 1) / kTilePos, all_blocks = (n + kBlockPos - 1) / kBlockPos;
    const uint32_t* table = p.batch.table + (size_t)seq * p.batch.stride;
    if (tid == 0) *bad_s = 0;
    uint32_t bad = 0, away = 0;
    __syncthreads();

    // ---- query digits into tensor memory: a thread's row, 32 elements.  A warp loads two rows at a
    // time, sixteen lanes along each, and turns them around in shared memory ([plane][pair][row]).
    {
      uint32_t* turn = reinterpret_cast<uint32_t*>(sm) + warp * (48 * 33);
      const uint32_t pair = lane & 15u;
      longlong2 words[16];
#pragma unroll
      for (uint32_t i = 0; i < 16; ++i) {
        // (rows behind the last repeat it, so that no branch comes between the loads)
        const uint32_t q = min(v0 + 32 * (warp & 3) + 2 * i + (lane >> 4), queries - 1), token = q / group;
        words[i] = __ldg(reinterpret_cast<const longlong2*>(p.q + (size_t)(sq.first + token) * p.q_stride +
                                                            (size_t)(kvh * group + q - token * group) * HD + 32 * cg) +
                         pair);
      }
#pragma unroll
      for (uint32_t i = 0; i < 16; ++i) {
        const uint32_t row = 2 * i + (lane >> 4);
        const longlong2 x = words[i];
        const uint64_t a = (uint64_t)x.x + 0x808080u, b = (uint64_t)x.y + 0x808080u;
        bad |= (uint32_t)((a | b) >> 24 != 0);
        const uint32_t u = __byte_perm((uint32_t)a, (uint32_t)b, 0x5410), t = __byte_perm((uint32_t)a, (uint32_t)b, 0x7632);
        turn[pair * 33 + row] = sub_1152(lift<0x4240>(u));
        turn[(16 + pair) * 33 + row] = sub_1152(lift<0x4341>(u));
        turn[(32 + pair) * 33 + row] = sub_1152(lift<0x4240>(t));
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = turn[(16 * k + i) * 33 + lane];
        tmem_st16(tmem + lane_base + k * (HD / 2) + 16 * cg, w);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      __syncthreads();  // the keys' operands go to the same place
      for (uint32_t i = tid; i < T::kKeys / 2 / 16; i += T::kThreads) {  // places 0, 1, 5, 6, 10 and 11
        const uint32_t half = i / (T::kKeyHalf / 2 / 16), in = i % (T::kKeyHalf / 2 / 16), at = in / (T::kKeyPlane / 16);
        *reinterpret_cast<uint4*>(sm + half * T::kKeyHalf + (at / 2 * 5 + at % 2) * T::kKeyPlane +
                                  in % (T::kKeyPlane / 16) * 16) = make_uint4(0, 0, 0, 0);
      }
    }

    // ---- scores: 32 positions at a time
    const uint32_t kpos = tid / (HD / 8), kchunk = tid % (HD / 8);
    int4 raw[2];
    uint32_t next_id = 0;
    auto page_of = [&](uint32_t at) {  // of position c0 + at
      return at < n ? __ldg(table + ((c0 + at) >> shift)) : CK_NO_PAGE;
    };
    auto load_keys = [&](uint32_t i) {  // by the page looked up before, and looks the next one up
      const uint32_t at = i * kTilePos + kpos, t = c0 + at, id = next_id;
      raw[0] = raw[1] = make_int4(0, 0, 0, 0);
      if (id < p.pool.pages) {
        const int4* src = reinterpret_cast<const int4*>(p.pool.k + page_word(p.pool, id, kvh) +
                                                        (size_t)(t & pmask) * HD + 8 * kchunk);
        raw[0] = __ldg(src);
        raw[1] = __ldg(src + 1);
      } else if (at < n && ((t & pmask) == 0 || at == 0)) {
        note(p.batch, seq, err_key((t >> shift) << shift, p.pool.layer, CK_PAGED_BAD_PAGE, 0));
      }
      next_id = page_of(at + kTilePos);
    };
    auto put_keys = [&](uint32_t buf) {
      const uint32_t y[8] = {biased(raw[0].x), biased(raw[0].y), biased(raw[0].z), biased(raw[0].w),
                             biased(raw[1].x), biased(raw[1].y), biased(raw[1].z), biased(raw[1].w)};
      uint32_t d[3][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = y[2 * i], b = y[2 * i + 1];
        bad |= (a | b) >> 24;
        const uint32_t u = __byte_perm(a, b, 0x5410), t = __byte_perm(a, b, 0x7632);
        d[0][i] = sub_1152(lift<0x4240>(u));
        d[1][i] = sub_1152(lift<0x4341>(u));
        d[2][i] = sub_1152(lift<0x4240>(t));
      }
      uint8_t* dst = sm + (kchunk >> 3) * T::kKeyHalf + (2 + 5 * buf) * T::kKeyPlane + kpos * 128 +
                     (((kchunk & 7u) ^ (kpos & 7u)) << 4);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint4*>(dst + k * T::kKeyPlane) = make_uint4(d[k][0], d[k][1], d[k][2], d[k][3]);
      fence_operands();
    };
    // A batch's products, by one thread of the warps in turn, once its operands are in place and
    // its accumulators drained.
    auto issue_scores = [&](uint32_t i) {
      if (warp_u == i % kWarps) {
        wait_full(batch + i);
        if (i >= T::kBufs) wait_drained(tiles + i - T::kBufs);
        const uint32_t leader = elected(), d0 = tmem_u + T::kScoreCol + (i % T::kBufs) * (kDiags * kTilePos);
        const uint64_t b0 = operands + ((2 + 5 * (i & 1u)) * T::kKeyPlane >> 4);
        // A query plane times five places side by side, the three key planes and zeros, adds to the
        // five accumulators at once: plane qp's begin qp places before the keys.  Products of one
        // shape into the same accumulators are done in order; of several shapes into parts of
        // them, which measured 234 against 249 us and 337 against 357, they need not be.
#pragma unroll
        for (uint32_t kk = 0; kk < HD / 16; ++kk)
#pragma unroll
          for (uint32_t qp = 0; qp < 3; ++qp)
            mma_ts(leader, d0, tmem_u + qp * (HD / 2) + 8 * kk,
                   b0 + ((kk >> 2) * T::kKeyHalf >> 4) - (qp * T::kKeyPlane >> 4) + 2 * (kk & 3u),
                   tile_idesc(kDiags * kTilePos), kk + qp != 0);
        commit(leader, done + ((batch + i) & 1u));
      }
      __syncwarp();
    };
    int32_t m = INT32_MIN;
    constexpr uint32_t kCols = kTilePos / T::kGroups;  // columns a thread drains
    auto drain_scores = [&](uint32_t i) {
      const uint32_t base = tmem + lane_base + T::kScoreCol + (i % T::kBufs) * (kDiags * kTilePos) + cg * kCols;
#pragma unroll
      for (uint32_t h = 0; h < kCols; h += 8) {
        uint32_t d[kDiags][8];
#pragma unroll
        for (uint32_t g = 0; g < kDiags; ++g) tmem_ld8(base + g * kTilePos + h, d[g]);
        tmem_wait_ld(d);
        const uint32_t at = i * kTilePos + cg * kCols + h;
        int32_t c[8];
        float high[8], peak = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          high[j] = fmaf(__uint_as_float(d[4][j]), 256.0f, __uint_as_float(d[3][j]));
          peak = fmaxf(peak, fabsf(high[j]));
          if (HD > 64) peak = fmaxf(peak, fabsf(__uint_as_float(d[2][j])));  // (3 * 64 * 2^14 < 2^22)
        }
        if (peak <= 4194304.0f && p.inv_sqrt <= 1u << 24) {
          // the usual case: the two highest accumulators join exactly, every number lies within
          // 2^22 and turns into an integer by an addition, (the sum of the accumulators by
          // weight) >> 16 fits 32 bits, and so the score
          constexpr uint32_t kOne = 0x4B400000u;  // the bits of kWhole; those of kWhole + x are x more
          constexpr float kWhole = 12582912.0f;   // 3 * 2^22
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t x0 = __float_as_uint(__uint_as_float(d[0][j]) + kWhole);
            const uint32_t x1 = __float_as_uint(__uint_as_float(d[1][j]) + kWhole);
            const uint32_t x2 = __float_as_uint(__uint_as_float(d[2][j]) + kWhole);
            const uint32_t x3 = __float_as_uint(high[j] + kWhole);
            const int32_t lo = (int32_t)(x0 + (x1 << 8) - (kOne + (kOne << 8)));
            const int32_t dot = (int32_t)((uint32_t)(lo >> 16) + x2 + (x3 << 8) - (kOne + (kOne << 8)));
            c[j] = (int32_t)(((int64_t)dot * (int32_t)p.inv_sqrt) >> 24);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int32_t lo = __float2int_rn(__uint_as_float(d[0][j])) + (__float2int_rn(__uint_as_float(d[1][j])) << 8);
            const int32_t mid = (lo >> 16) + __float2int_rn(__uint_as_float(d[2][j])) +
                                (__float2int_rn(__uint_as_float(d[3][j])) << 8);
            const int64_t dot = (int64_t)mid + ((int64_t)__float2int_rn(__uint_as_float(d[4][j])) << 16);
            const int64_t s = wmul(dot, (int64_t)p.inv_sqrt) >> 24;
            c[j] = (int32_t)s;
            if (c[j] != s) c[j] = s < 0 ? INT32_MIN : INT32_MAX;
          }
        }
        if (at + 8 <= lim) {
#pragma unroll
          for (int j = 0; j < 8; ++j) m = max(m, c[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (at + j < lim) m = max(m, c[j]);
        }
        int4* dst = scores + (size_t)(at / 4) * kTileRows + r;
        dst[0] = make_int4(c[0], c[1], c[2], c[3]);
        dst[kTileRows] = make_int4(c[4], c[5], c[6], c[7]);
      }
    };
    if (nt) {
      next_id = page_of(kpos);
      load_keys(0);
      put_keys(0);
      arrive(full + (batch & 1u));
      load_keys(1);
      issue_scores(0);
    }
    for (uint32_t i = 0; i < nt; ++i) {
      if (i + 1 < nt) {
        put_keys((i + 1) & 1u);  // (the products that read the place before are done: tile i - 1's)
        arrive(full + ((batch + i + 1) & 1u));
        load_keys(i + 2);
        if (T::kBufs == 2) issue_scores(i + 1);
      }
      wait_done(batch + i);
      drain_scores(i);
      arrive(drained + ((tiles + i) & 1u));
      if (T::kBufs == 1 && i + 1 < nt) issue_scores(i + 1);
    }
    batch += nt;
    tiles += nt;
    asm volatile("fence.proxy.async.global;" ::: "memory");  // the scores come back by bulk copies

    // ---- the row's maximum, over the column groups and the cluster
    int32_t* redm = reinterpret_cast<int32_t*>(red);
    redm[cg * kTileRows + r] = m;
    if (bad) *bad_s = 1;
    __syncthreads();
    if (tid < kTileRows) {
      for (uint32_t g = 1; g < T::kGroups; ++g) m = max(m, redm[g * kTileRows + tid]);
      xmax[tid] = m;
    }
    all_sync(C);
    m = xmax[r];
    away = *bad_s;
    if (C > 1) {
      int32_t peak[8];
      uint32_t flag[8];
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {
        peak[k] = k < C ? (int32_t)peer32(xmax + r, k) : INT32_MIN;
        flag[k] = k < C ? peer32(bad_s, k) : 0;
      }
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {
        m = max(m, peak[k]);
        away |= flag[k];
      }
    }
    // a maximum at either end of 32 bits: a score may have been cut that counts
    away |= (uint32_t)(np != 0 && (m == INT32_MAX || m < INT32_MIN + (1 << 21)));
    away = (uint32_t)__syncthreads_or((int)away);  // (the same rows, so the same in every block)

    // ---- the exponentials, in the place of the scores, and their sum
    unsigned long long z = 0;
    if (!away) {
      constexpr uint32_t kMine = kTilePos / 4 / T::kGroups;  // quads of a stage a thread takes
      auto fetch = [&](uint32_t i) {  // by one thread
        const uint32_t at = (staged + i) % kRing;
        mb_expect_tx(ring + at, kStage);
        bulk_copy(sm + at * kStage, scores + (size_t)i * (kStage / 16), kStage, ring + at);
      };
      if (tid == 0)
        for (uint32_t i = 0; i < min(nt, kRing); ++i) fetch(i);
      for (uint32_t i = 0; i < nt; ++i) {
        const uint32_t at = staged + i;
        if (tid == 0 && i > 0 && i - 1 + kRing < nt) {
          wait_copy(freed + (at - 1) % kRing, ((at - 1) / kRing) & 1u);
          fetch(i - 1 + kRing);
        }
        wait_copy(ring + at % kRing, (at / kRing) & 1u);
        const int4* stage = reinterpret_cast<const int4*>(sm + (at % kRing) * kStage) + r;
        int4 c[kMine];
#pragma unroll
        for (uint32_t u = 0; u < kMine; ++u) c[u] = stage[(cg + T::kGroups * u) * kTileRows];
#pragma unroll
        for (uint32_t u = 0; u < kMine; ++u) {
          const uint32_t k = i * (kTilePos / 4) + cg + T::kGroups * u;
          const int32_t x[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
          uint32_t e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = table_s[min(((uint32_t)m - (uint32_t)x[j]) >> 8, 4096u)];
          if (4 * k + 4 > lim) {  // the last quad may be cut
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (4 * k + j >= lim) e[j] = 0;
          }
          if (4 * k < lim) {
            z += (unsigned long long)(e[0] + e[1]) + (e[2] + e[3]);
            scores[(size_t)k * kTileRows + r] = make_int4(e[0], e[1], e[2], e[3]);
          }
        }
        // Only now, as the lookups above needed the words: neither a barrier of the block nor an
        // arrival holds back the next copy until reads on their way have come.
        __syncwarp();
        if (lane == 0) mb_arrive(freed + at % kRing);
      }
      staged += nt;
    }
    red[cg * kTileRows + r] = z;
    __syncthreads();
    if (tid < kTileRows) {
      for (uint32_t g = 1; g < T::kGroups; ++g) z += red[g * kTileRows + tid];
      xsum[tid] = z;
    }
    all_sync(C);
    z = xsum[r];
    if (C > 1) {
      unsigned long long part[8];
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) part[k] = k < C ? peer64(xsum + r, k) : 0;
      z = 0;
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) z += part[k];
    }
    if (z < (1ull << 30)) z = 1ull << 30;
    const bool alone = z <= 1ull << 30;  // one score counts: P = e >> 6, and it may be 2^24
    const uint32_t rz = alone ? 0u : (uint32_t)div_by_estimate(1ull << 62, z, rcp_estimate((float)z));

    // ---- weighted values: 64 positions at a time
    const uint32_t nb = away ? 0 : all_blocks;
    const uint32_t vchunk = tid & 7u, vpair = tid >> 3;  // eight positions, two elements
    constexpr uint32_t kChunks = 8 / T::kGroups;         // chunks of eight scores a thread takes
    int2 vraw[8];
    int4 sraw[2 * kChunks];
    auto load_values = [&](uint32_t b) {
      const uint32_t at = b * kBlockPos + vchunk * 8, t = c0 + at, id = next_id;
#pragma unroll
      for (int j = 0; j < 8; ++j) vraw[j] = make_int2(0, 0);
      if (id < p.pool.pages) {  // a page holds whole chunks of eight
        const int2* src = reinterpret_cast<const int2*>(p.pool.v + page_word(p.pool, id, kvh) +
                                                        (size_t)(t & pmask) * HD + 2 * vpair);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at + j < n) vraw[j] = __ldg(src + j * (HD / 2));
      }
      next_id = page_of(at + kBlockPos);
    };
    auto load_scores = [&](uint32_t b) {
#pragma unroll
      for (uint32_t c = 0; c < kChunks; ++c) {
        const uint32_t at = b * kBlockPos + (cg * kChunks + c) * 8;
        const int4* src = scores + (size_t)(at / 4) * kTileRows + r;
        sraw[2 * c] = at < lim ? src[0] : make_int4(0, 0, 0, 0);
        sraw[2 * c + 1] = at + 4 < lim ? src[kTileRows] : make_int4(0, 0, 0, 0);
      }
    };
    auto put_values = [&](uint8_t* planes) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t d[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a = biased(e ? vraw[2 * i].y : vraw[2 * i].x);
          const uint32_t b = biased(e ? vraw[2 * i + 1].y : vraw[2 * i + 1].x);
          bad |= (a | b) >> 24;
          const uint32_t u = __byte_perm(a, b, 0x5410), t = __byte_perm(a, b, 0x7632);
          d[0][i] = fma_h2(lift<0x4240>(u), kScale0, kBal0);
          d[1][i] = fma_h2(lift<0x4341>(u), kScale1, kBal1);
          d[2][i] = fma_h2(lift<0x4240>(t), kScale2, kBal2);
        }
        const uint32_t row = 2 * vpair + e;
        uint8_t* dst = planes + row * 128 + ((vchunk ^ (row & 7u)) << 4);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4*>(dst + k * T::kValuePlane) = make_uint4(d[k][0], d[k][1], d[k][2], d[k][3]);
      }
    };
    auto put_probs = [&](uint32_t b, uint8_t* planes) {
#pragma unroll
      for (uint32_t c = 0; c < kChunks; ++c) {
        const uint32_t chunk = cg * kChunks + c, at = b * kBlockPos + chunk * 8;
        const int4 s0 = sraw[2 * c], s1 = sraw[2 * c + 1];
        const uint32_t s[8] = {(uint32_t)s0.x, (uint32_t)s0.y, (uint32_t)s0.z, (uint32_t)s0.w,
                               (uint32_t)s1.x, (uint32_t)s1.y, (uint32_t)s1.z, (uint32_t)s1.w};
        uint32_t pr[8], differ = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t e = s[j];
          // floor((e << 24) / z): with rz = floor(2^62 / z) it lies between the products of e with
          // rz and rz + 1, >> 38; where those differ (less than one in 2^8) the remainder decides
          const uint32_t low = __umulhi(e, rz), high = __umulhi(e, rz + 1);
          pr[j] = low >> 6;
          differ |= low ^ high;
        }
        if (differ >> 6) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const unsigned long long rem = ((unsigned long long)s[j] << 24) - (unsigned long long)pr[j] * z;
            pr[j] += rem >= z;
          }
        }
        if (alone) {
#pragma unroll
          for (int j = 0; j < 8; ++j) pr[j] = s[j] >> 6;
        }
        uint32_t d[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a = pr[2 * i], bq = pr[2 * i + 1], extra = 0;
          if (alone) {  // P = 2^24 is 0xFFFFFF and one more in the lowest digit (2^-12 in its plane)
            extra = (a >> 24 ? 0x0C00u : 0u) | (bq >> 24 ? 0x0C000000u : 0u);
            a -= a >> 24;
            bq -= bq >> 24;
          }
          const uint32_t u = __byte_perm(a, bq, 0x5410), t = __byte_perm(a, bq, 0x7632);
          d[0][i] = fma_h2(lift<0x4240>(u), kScale0, kUns0);
          d[1][i] = fma_h2(lift<0x4341>(u), kScale1, kUns1);
          d[2][i] = fma_h2(lift<0x4240>(t), kScale2, kUns2);
          if (alone) asm("add.rn.f16x2 %0, %0, %1;" : "+r"(d[0][i]) : "r"(extra));
        }
        uint8_t* dst = planes + r * 128 + ((chunk ^ (r & 7u)) << 4);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4*>(dst + k * T::kProbPlane) = make_uint4(d[k][0], d[k][1], d[k][2], d[k][3]);
      }
    };
    // Adds the accumulators to the 64-bit sums, which lie in the scratch between flushes; the
    // last flush leaves them in shared memory, [element][row].
    unsigned long long* sums = reinterpret_cast<unsigned long long*>(sm);
    auto flush = [&](bool first, bool final) {
#pragma unroll
      for (uint32_t h = 0; h < 32; h += 8) {
        unsigned long long old[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) old[j] = final && !first ? __ldcg(kept + (h + j) * T::kThreads) : 0;
        uint32_t d[4][8];
#pragma unroll
        for (uint32_t g = 0; g < 4; ++g) tmem_ld8(tmem + lane_base + g * HD + 32 * cg + h, d[g]);
        tmem_wait_ld(d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          long long t = __float2int_rn(__uint_as_float(d[0][j]) * 16777216.0f);
          t += (long long)__float2int_rn(__uint_as_float(d[1][j]) * 65536.0f) * 256;
          t += (long long)__float2int_rn(__uint_as_float(d[2][j]) * 256.0f) * 65536;
          t += (long long)__float2int_rn(__uint_as_float(d[3][j])) * 16777216;
          if (final)
            sums[(size_t)(32 * cg + h + j) * T::kPitch + r] = (unsigned long long)t + old[j];
          else if (first)
            __stcg(kept + (h + j) * T::kThreads, (unsigned long long)t);
          else
            atomicAdd(kept + (h + j) * T::kThreads, (unsigned long long)t);  // nothing to wait for
        }
      }
    };
    auto issue_values = [&](uint32_t b) {
      if (warp_u == b % kWarps) {
        wait_full(batch + b);
        const uint32_t leader = elected();
        const uint64_t a0 = operands + (b % T::kBufs) * (T::kValueBuf >> 4), b0 = a0 + (3 * T::kProbPlane >> 4);
        const uint32_t go_on = b % kFlushBlocks != 0;
        // The products of a weight have one shape and their accumulator to themselves; that of the
        // highest weight shares the last.
#pragma unroll
        for (uint32_t kk = 0; kk < kBlockPos / 16; ++kk)
#pragma unroll
          for (uint32_t pp = 0; pp < 3; ++pp)
#pragma unroll
            for (uint32_t vp = 0; vp < 3; ++vp) {
              const uint32_t g = min(pp + vp, 3u);
              const bool begins = kk == 0 && (pp == 0 || (pp == 1 && vp == 2));
              mma_ss(leader, tmem_u + g * HD, a0 + ((pp * T::kProbPlane + kk * 32) >> 4),
                     b0 + ((vp * T::kValuePlane + kk * 32) >> 4), tile_idesc(HD), begins ? go_on : 1u);
            }
        commit(leader, done + ((batch + b) & 1u));
      }
      __syncwarp();
    };
    if (nb) {
      next_id = page_of(vchunk * 8);
      load_values(0);
      load_scores(0);
    }
    for (uint32_t b = 0; b < nb; ++b) {
      uint8_t* planes = sm + (b % T::kBufs) * T::kValueBuf;
      if (b >= T::kBufs) wait_done(batch + b - T::kBufs);  // the place is free
      put_values(planes + 3 * T::kProbPlane);
      load_values(b + 1);
      put_probs(b, planes);
      if (b + 1 < nb) load_scores(b + 1);
      fence_operands();
      if (b > 0 && b % kFlushBlocks == 0) {
        wait_done(batch + b - 1);
        flush(b == kFlushBlocks, false);
      }
      arrive(full + ((batch + b) & 1u));
      issue_values(b);
    }
    if (T::kBufs == 2 && nb > 1) wait_done(batch + nb - 2);  // (another thread's products)
    if (nb) wait_done(batch + nb - 1);
    batch += nb;
    if (bad) *bad_s = 1;
    if (tid == 0 && *abort_flag) *bad_s = 1;
    __syncthreads();  // every warp has seen the last products done: they read the sums' place

    // ---- the cluster's sums, a slice of the rows each block
    if (nb) {
      flush(nb <= kFlushBlocks, true);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) sums[(size_t)(32 * cg + j) * T::kPitch + r] = 0;
    }
    all_sync(C);
    away |= *bad_s;
    for (uint32_t k = 0; C > 1 && k < C; ++k) away |= peer32(bad_s, k);
    const uint32_t then = C > 1 ? peer32(next_s, 0) : *next_s;
    const uint32_t rows = kTileRows / C;
    for (uint32_t i = tid; !away && i < rows * HD; i += T::kThreads) {
      const uint32_t row = rank * rows + i / HD, e = i % HD, q = v0 + row;
      if (q >= queries) break;
      unsigned long long t = 0;
      if (C > 1) {
        unsigned long long part[8];
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) part[k] = k < C ? peer64(sums + (size_t)e * T::kPitch + row, k) : 0;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) t += part[k];
      } else {
        t = sums[(size_t)e * T::kPitch + row];
      }
      p.out[((size_t)(sq.first + q / group) * p.heads + kvh * group + q % group) * HD + e] = (long long)t >> 24;
    }
    if (rank == 0 && tid == 0) {
      f.away[item] = away;
      if (away) atomicAdd(f.any, 1u);
    }
    all_sync(C);  // no block goes on while another reads its sums or flags
    item = then;
  }
  tc_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(T::kTmem) : "memory");
}

template <int HD>
cudaError_t configure_tiles(const DeviceFacts& f) {
  static std::atomic<bool> ready[64];
  if (ready[f.dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(k_pattn_tiles<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tile<HD>::kSmem);
  if (e == cudaSuccess) ready[f.dev].store(true, std::memory_order_relaxed);
  return e;
}

template <int HD>
void tiles_config(uint32_t blocks, uint32_t C, cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr) {
  *cfg = {};
  cfg->gridDim = dim3(blocks);
  cfg->blockDim = dim3(Tile<HD>::kThreads);
  cfg->dynamicSmemBytes = Tile<HD>::kSmem;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = C;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

// Clusters of C blocks that are resident at once, looked up once for each C (the runtime counts one
// block an SM; of head size 64 two run).  0 where the lookup fails: no plan then uses that C, and the
// failure is not left for a later call to report.
template <int HD>
int32_t resident_clusters(uint32_t C, const DeviceFacts& f) {
  static std::atomic<int> known[64][9];  // the number and one more, zero before
  int n = known[f.dev][C].load(std::memory_order_relaxed) - 1;
  if (n < 0) {
    cudaError_t e = configure_tiles<HD>(f);
    if (e == cudaSuccess) {
      cudaLaunchConfig_t cfg;
      cudaLaunchAttribute attr[1];
      tiles_config<HD>(C, C, &cfg, attr);
      e = cudaOccupancyMaxActiveClusters(&n, k_pattn_tiles<HD>, &cfg);
    }
    if (e != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    n *= HD == 64 ? 2 : 1;
    known[f.dev][C].store(n + 1, std::memory_order_relaxed);
  }
  return n;
}

template <int HD>
cudaError_t launch_tiles_hd(const TilesParams& p, const TilesPlan& w, const DeviceFacts& f, cudaStream_t s) {
  const cudaError_t e = configure_tiles<HD>(f);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  tiles_config<HD>(w.clusters * w.C, w.C, &cfg, attr);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, k_pattn_tiles<HD>, p);
}

}  // namespace

bool tiles_fit(const ck_paged_cache& c, const DeviceFacts& f) {
  return (c.head_dim == 64 && Tile<64>::kSmem <= (uint32_t)f.optin) ||
         (c.head_dim == 128 && Tile<128>::kSmem <= (uint32_t)f.optin);
}

void resident_tiles(const ck_paged_cache& c, const DeviceFacts& f, int32_t* out) {
  for (int i = 0; i < kTileClusters; ++i)
    out[i] = !tiles_fit(c, f) ? 0 : c.head_dim == 64 ? resident_clusters<64>(1u << i, f) : resident_clusters<128>(1u << i, f);
}

TilesPlan plan_tiles(const ck_paged_cache& c, const ck_paged_batch& b, uint32_t heads, const DeviceFacts& f,
                     const int32_t* resident) {
  TilesPlan w = {};
  const uint64_t queries = (uint64_t)b.max_new * (heads / c.kv_heads);
  if (!tiles_fit(c, f)) return w;
  w.tiles = (uint32_t)((queries + kTileRows - 1) / kTileRows);
  const uint64_t items = (uint64_t)b.seqs * c.kv_heads * w.tiles;
  if (items > 0xFFFFFFFFull - 65536) return w;  // (the count of tiles is 32 bits)
  // Blocks of a cluster, by what each choice takes, in positions a block goes through: rounds of
  // equal tiles for one sequence; for several, whose lengths differ, three quarters of the bound
  // on average, but never less than the longest.  What surrounds a tile (queries, exchanges,
  // sums) measured as about 200 positions.
  double best = 0;
  for (int i = 0; i < kTileClusters; ++i) {
    if (resident[i] <= 0) continue;
    const uint32_t C = 1u << i;
    const double each = (double)b.max_len / C + 200, clusters = (double)std::min<uint64_t>(items, resident[i]);
    const double cost = b.seqs == 1 ? std::ceil(items / clusters) * each
                                    : std::max(each, items / clusters * (0.75 * b.max_len / C + 200));
    if (!w.use || cost < 0.95 * best) {
      w.use = true;
      best = cost;
      w.C = C;
      w.clusters = (uint32_t)clusters;
    }
  }
  if (!w.use) return w;
  w.cap = ((b.max_len + w.C - 1) / w.C + kBlockPos - 1) & ~(kBlockPos - 1);
  w.any_off = 0;
  w.away_off = 256;
  w.scores_off = w.away_off + align256(4 * items);
  w.sums_off = w.scores_off + align256(4ull * kTileRows * w.cap * w.clusters * w.C);
  w.size = w.sums_off + 8ull * kTileRows * c.head_dim * w.clusters * w.C;
  return w;
}

cudaError_t launch_tiles(const TilesParams& p, const TilesPlan& w, const DeviceFacts& f, cudaStream_t s) {
  return p.a.pool.hd == 64 ? launch_tiles_hd<64>(p, w, f, s) : launch_tiles_hd<128>(p, w, f, s);
}

}  // namespace ck

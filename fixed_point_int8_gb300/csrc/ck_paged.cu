// The paged cache's stores and its page tables ("The attention cache"; "The forward pass, in
// order", phases 6 to 8): rotary with checked stores into pages, and forking, growing, freeing
// and packing of the tables with the copies of pages that they need.
#include "ck_paged.cuh"

namespace ck {
namespace {

// ------------------------------------------------------------------ rotary and stores

struct StoreParams {
  PoolView pool;
  BatchView batch;
  const int64_t* q;
  const int64_t* k;
  const int64_t* v;
  size_t q_stride, k_stride, v_stride;
  uint32_t heads, rope_rows, rot, half;
  const int32_t* rope;
  int64_t* q_out;
};

constexpr int kStoreThreads = 256;

__device__ __forceinline__ void load2(const int64_t* p, int64_t& a, int64_t& b) {
  const longlong2 w = *reinterpret_cast<const longlong2*>(p);
  a = w.x;
  b = w.y;
}

// Row blockIdx.x; a unit is four elements of a head of the queries, keys or values: in the half
// layout two pairs (j, j + rot / 2) and (j + 1, j + 1 + rot / 2), otherwise four in a row.  A
// thread takes unit after unit, gridDim.y blocks' threads apart, the next one's words under way:
// one block a row where rows fill the GPU (looking up a row's sequence and page for every 256
// units took 29.5 us for 1,600 rows of 6,144 elements, once a row 26.2), a unit a thread where
// they do not.  The instructions bound it (over 200 a unit with a turned pair's 64-bit products,
// checks and addresses: 63 % of the issue slots), with half of the warps resident at 58 registers.
__global__ void __launch_bounds__(kStoreThreads) k_paged_store(const StoreParams p) {
  const uint32_t row = blockIdx.x, hd = p.pool.hd;
  const uint32_t shift = 31 - __clz((int)hd) - 2, kvh = p.pool.kv_heads;  // log2 of a head's units
  const uint32_t units = (p.heads + 2 * kvh) << shift, step = gridDim.y * kStoreThreads;
  uint32_t unit = blockIdx.y * kStoreThreads + threadIdx.x;
  struct Unit {
    uint32_t head, e0, e1;  // its elements: e0, e0 + 1 and e1, e1 + 1
    bool is_q, is_v, turned, halves;
    int64_t x[4];
  };
  auto load = [&](uint32_t n) {
    Unit w;
    w.head = n >> shift;
    const uint32_t u = n & ((1u << shift) - 1);
    w.is_q = w.head < p.heads;
    w.is_v = w.head >= p.heads + kvh;
    w.head -= w.is_q ? 0u : w.is_v ? p.heads + kvh : p.heads;
    w.turned = !w.is_v && 4 * u < p.rot;
    w.halves = w.turned && p.half;
    w.e0 = w.halves ? 2 * u : 4 * u;
    w.e1 = w.halves ? 2 * u + p.rot / 2 : 4 * u + 2;
    if (n < units) {
      const int64_t* src = (w.is_q ? p.q + row * p.q_stride : w.is_v ? p.v + row * p.v_stride : p.k + row * p.k_stride) +
                           w.head * hd;
      load2(src + w.e0, w.x[0], w.x[1]);
      load2(src + w.e1, w.x[2], w.x[3]);
    }
    return w;
  };
  Unit w = load(unit);  // (asked for before the sequence is looked up)
  const uint32_t s = block_find_seq(p.batch, row);
  if (s >= p.batch.seqs) return;
  const Sequence sq = load_sequence(p.batch, s, p.pool.page_shift);
  if (row < sq.first) return;  // before the first sequence
  const bool lead = unit == 0;
  if (!sq.ok) {
    if (lead) note(p.batch, s, err_key(0, p.pool.layer, CK_PAGED_BAD_SEQUENCE, 0));
    return;
  }
  if (!sq.holds(row)) return;
  const uint32_t up = row - sq.first + sq.len;  // position + count
  if (up < sq.count) return;
  const uint32_t pos = up - sq.count;
  if (p.rot != 0 && pos >= p.rope_rows) {
    if (lead) note(p.batch, s, err_key(pos, p.pool.layer, CK_PAGED_BAD_SEQUENCE, 0));
    return;
  }
  const uint32_t id = p.batch.table[(size_t)s * p.batch.stride + (pos >> p.pool.page_shift)];
  const bool paged = id < p.pool.pages;
  if (!paged && lead) note(p.batch, s, err_key(pos, p.pool.layer, CK_PAGED_BAD_PAGE, 0));
  const size_t slot = page_word(p.pool, paged ? id : 0, 0) + (size_t)(pos & ((1u << p.pool.page_shift) - 1)) * hd;
  const uint32_t head_words = hd << p.pool.page_shift;
  const int32_t* rope = p.rope + (size_t)pos * p.rot;
  int64_t* q_out = p.q_out + (size_t)row * p.heads * hd;
  while (unit < units) {
    // pair j of the table row: 2u and 2u + 1 of a head's unit u in both layouts
    int4 cs = make_int4(0, 0, 0, 0);
    if (w.turned) cs = __ldg(reinterpret_cast<const int4*>(rope + 4 * (unit & ((1u << shift) - 1))));
    const uint32_t next = unit + step;
    const Unit then = load(next);
    auto check = [&](uint32_t phase) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!fits_i32(w.x[i]))
          note(p.batch, s, err_key(pos, p.pool.layer, phase, w.head * hd + (i < 2 ? w.e0 + i : w.e1 + i - 2)));
    };
    if (!w.is_q) {
      check(w.is_v ? 7 : 6);
#pragma unroll
      for (int i = 0; i < 4; ++i) w.x[i] = (int32_t)w.x[i];
    }
    if (w.turned) {
      if (w.halves) {
        rotate_pair(w.x[0], w.x[2], cs.x, cs.y, w.x[0], w.x[2]);
        rotate_pair(w.x[1], w.x[3], cs.z, cs.w, w.x[1], w.x[3]);
      } else {
        rotate_pair(w.x[0], w.x[1], cs.x, cs.y, w.x[0], w.x[1]);
        rotate_pair(w.x[2], w.x[3], cs.z, cs.w, w.x[2], w.x[3]);
      }
    }
    if (w.is_q) {
      int64_t* dst = q_out + w.head * hd;
      *reinterpret_cast<longlong2*>(dst + w.e0) = make_longlong2(w.x[0], w.x[1]);
      *reinterpret_cast<longlong2*>(dst + w.e1) = make_longlong2(w.x[2], w.x[3]);
    } else {
      if (w.turned) check(8);
      if (paged) {
        int32_t* dst = (w.is_v ? p.pool.v : p.pool.k) + slot + (size_t)w.head * head_words;
        *reinterpret_cast<int2*>(dst + w.e0) = make_int2((int32_t)w.x[0], (int32_t)w.x[1]);
        *reinterpret_cast<int2*>(dst + w.e1) = make_int2((int32_t)w.x[2], (int32_t)w.x[3]);
      }
    }
    unit = next;
    w = then;
  }
}

// ------------------------------------------------------------------ page tables

struct Copy {
  uint32_t src, dst, count, pad;  // count: filled positions
};

// Scratch of a call, from 256-byte aligned offsets.  [0, zero) is cleared first.
struct PagesLayout {
  uint64_t owner, bits, counters, zero, list, list2, before, copies, size;
};
PagesLayout pages_layout(uint32_t pages, uint32_t rows) {
  PagesLayout w;
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) { uint64_t o = off; off = align256(off + bytes); return o; };
  w.owner = take(4ull * pages);
  w.bits = take(4ull * ((pages + 31) / 32));
  w.counters = take(256);
  w.zero = off;
  w.list = take(4ull * pages);
  w.list2 = take(4ull * pages);
  w.before = take(8ull * rows);
  w.copies = take(sizeof(Copy) * (uint64_t)std::max(pages, rows));
  w.size = off;
  return w;
}

// The listed copies of pages, keys and values: warp `first` of `warps`, then every one `warps`
// on, takes one head's filled positions of one layer, count * head_dim words in a row.  HBM bounds
// it: packing 1.5 GB takes 234 us (6.4 TB/s); runs of 2 KB, where a fork copies a few positions a
// page, reach 5.1 TB/s.
constexpr uint32_t kCopyAhead = 8;
struct CopyJob {
  int32_t* k;
  int32_t* v;
  uint32_t runs, page_shift, hd;
};
__device__ __forceinline__ void copy_pages(const CopyJob& c, const Copy* copies, uint32_t count, uint64_t first,
                                           uint64_t warps) {
  const uint32_t lane = threadIdx.x & 31;
  const uint64_t tasks = 2ull * c.runs * count;
  const uint32_t page4 = (c.hd << c.page_shift) / 4;  // 16-byte words of a head's page
  for (uint64_t t = first; t < tasks; t += warps) {
    const uint64_t i = t / (2 * c.runs);
    const uint32_t rest = (uint32_t)(t - i * 2 * c.runs), run = rest >> 1;
    const Copy one = copies[i];
    int4* pool = reinterpret_cast<int4*>(rest & 1 ? c.v : c.k);
    const int4* src = pool + ((size_t)one.src * c.runs + run) * page4;
    int4* dst = pool + ((size_t)one.dst * c.runs + run) * page4;
    const uint32_t n = one.count * (c.hd / 4);
    for (uint32_t j0 = lane; j0 < n; j0 += 32 * kCopyAhead) {  // loads in flight before the stores
      int4 w[kCopyAhead];
#pragma unroll
      for (uint32_t u = 0; u < kCopyAhead; ++u)
        if (j0 + 32 * u < n) w[u] = __ldcs(src + j0 + 32 * u);
#pragma unroll
      for (uint32_t u = 0; u < kCopyAhead; ++u)
        if (j0 + 32 * u < n) __stcs(dst + j0 + 32 * u, w[u]);
    }
  }
}
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads) k_copy_pages(const CopyJob c, const Copy* copies, const uint32_t* count) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  copy_pages(c, copies, *count, (uint64_t)blockIdx.x * (kCopyThreads / 32) + threadIdx.x / 32,
             (uint64_t)gridDim.x * (kCopyThreads / 32));
}

struct PagesParams {
  const uint32_t* len_in;
  const uint32_t* table_in;
  const uint32_t* parent;
  const uint32_t* grow;
  const uint8_t* held;
  uint32_t* len_out;
  uint32_t* table_out;
  uint32_t* status;
  uint32_t* used_out;
  uint32_t rows_in, rows, stride, pages, page_shift, sinks, window;
  uint32_t* owner;      // pages: rows - the lowest row that holds the page part-filled (0: none)
  uint32_t* bits;       // pages that a row holds whole (packing: holds at all)
  uint32_t* copied;     // number of copies
  uint32_t* list;
  uint32_t* list2;
  unsigned long long* before;
  Copy* copies;
};

constexpr int kTableThreads = 256;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ bool bit_of(const uint32_t* bits, uint32_t i) { return (bits[i >> 5] >> (i & 31)) & 1u; }

// Of a sequence of `len` positions on `have` pages the ones that its next position or a later one sees: those
// with a position below `sinks`, and from the one on that ends behind len - window.  The page that the next
// position goes on in is one of them, whatever the window.
struct Kept {
  uint32_t early, late, have;
  __device__ __forceinline__ bool operator()(uint32_t i) const { return i < early || i - late < have - late; }
};
__device__ __forceinline__ Kept kept_pages(uint32_t len, uint32_t have, uint32_t sinks, uint32_t window, uint32_t page_shift) {
  const uint32_t early = (uint32_t)min(((unsigned long long)sinks + (1u << page_shift) - 1) >> page_shift, (unsigned long long)have);
  return {early, min(have, window <= len ? (len + 1 - window) >> page_shift : 0), have};
}

// Forking, first step (a warp a row): checks the row, takes over those of the parent's whole pages that its
// window keeps and marks them, and bids for its part-filled page.
__device__ __forceinline__ void fork_mark(const PagesParams& p, uint32_t r, uint32_t lane) {
  const uint32_t parent = p.parent[r];
  uint32_t status = 0, old = 0;
  if (parent != CK_NO_PAGE) {
    if (parent >= p.rows_in) {
      status = CK_INVALID_STATE;
    } else {
      old = p.len_in[parent];
      const uint64_t len = (uint64_t)old + p.grow[r];
      if (len > kMaxPositions || len > ((uint64_t)p.stride << p.page_shift)) status = CK_CONTEXT_EXCEEDED;
    }
  }
  const uint32_t full = old >> p.page_shift, part = old & ((1u << p.page_shift) - 1);
  const uint32_t* from = p.table_in + (size_t)parent * p.stride;
  const Kept keeps = kept_pages(old, full + (part != 0), p.sinks, p.window, p.page_shift);
  if (status == 0 && parent != CK_NO_PAGE) {
    bool bad = false;
    for (uint32_t i = lane; i < keeps.have; i += 32) bad |= keeps(i) && from[i] >= p.pages;
    if (__any_sync(0xffffffffu, bad)) status = CK_INVALID_STATE;
  }
  const bool live = status == 0 && parent != CK_NO_PAGE;
  uint32_t* to = p.table_out + (size_t)r * p.stride;
  for (uint32_t i = lane; i < p.stride; i += 32) {
    const uint32_t id = live && i < full && keeps(i) ? from[i] : CK_NO_PAGE;
    to[i] = id;
    if (id != CK_NO_PAGE) atomicOr(p.bits + (id >> 5), 1u << (id & 31));
  }
  if (lane == 0) {
    p.status[r] = status;
    p.len_out[r] = live ? old : CK_NO_PAGE;  // the old length, for the next step
    if (live && part) atomicMax(p.owner + from[full], p.rows - r);
  }
}
__global__ void __launch_bounds__(kTableThreads) k_fork_mark(const PagesParams p) {
  const uint32_t r = blockIdx.x * (kTableThreads / 32) + threadIdx.x / 32;
  if (r < p.rows) fork_mark(p, r, threadIdx.x & 31);
}

// Small calls do the steps before the copies in one block: clears the marks.
__device__ __forceinline__ void clear_marks(const PagesParams& p) {
  for (uint32_t i = threadIdx.x; i < p.pages; i += kPlanThreads) p.owner[i] = 0;
  for (uint32_t i = threadIdx.x; i < (p.pages + 31) / 32; i += kPlanThreads) p.bits[i] = 0;
  __syncthreads();
}

// Inclusive sum over the block's warps of one value a thread; *total the block's sum.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* warp_sum,
                                                         unsigned long long* total) {
  // (known to be the same in the warp: else the scan below, in a branch, collects the lanes at every step)
  const uint32_t lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const unsigned long long inc = warp_inclusive_scan(v, lane);
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  if (warp == 0) warp_sum[lane] = warp_inclusive_scan(warp_sum[lane], lane);
  __syncthreads();
  const unsigned long long base = warp ? warp_sum[warp - 1] : 0ull;
  *total = warp_sum[kPlanThreads / 32 - 1];
  __syncthreads();
  return base + inc;
}

// Second step (one block): what each row needs, the free pages in ascending order, and the
// rows' new pages and copies.  ALONE: with the first step before it.
template <bool ALONE>
__global__ void __launch_bounds__(kPlanThreads) k_fork_plan(const PagesParams p, const CopyJob job) {
  __shared__ unsigned long long warp_sum[kPlanThreads / 32];
  __shared__ uint32_t n_copies;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the copies wait for this grid's end)
  if (ALONE) {
    clear_marks(p);
    for (uint32_t r = warp; r < p.rows; r += kPlanThreads / 32) fork_mark(p, r, lane);
    __syncthreads();
  }
  const uint32_t mask = (1u << p.page_shift) - 1;
  if (tid == 0) n_copies = 0;
  // whether the row keeps its parent's part-filled page: as the lowest row that holds it, and where
  // no row holds it whole and no sequence outside the call has it
  auto stays = [&](uint32_t r, uint32_t old, uint32_t* last) {
    *last = p.table_in[(size_t)p.parent[r] * p.stride + (old >> p.page_shift)];
    return p.owner[*last] == p.rows - r && !bit_of(p.bits, *last) && !(p.held && (p.held[*last] & CK_PAGE_SHARED));
  };
  unsigned long long asked = 0;
  for (uint32_t base = 0; base < p.rows; base += kPlanThreads) {
    const uint32_t r = base + tid;
    unsigned long long need = 0;
    if (r < p.rows && p.len_out[r] != CK_NO_PAGE) {
      const uint32_t old = p.len_out[r], len = old + p.grow[r];
      uint32_t last;
      const uint32_t have = (old >> p.page_shift) + ((old & mask) && stays(r, old, &last) ? 1u : 0u);
      need = ((len + mask) >> p.page_shift) - have;
    }
    unsigned long long total;
    const unsigned long long end = asked + block_scan(need, warp_sum, &total);
    if (r < p.rows) p.before[r] = end - need;
    asked += total;
  }
  unsigned long long found = 0;
  for (uint32_t base = 0; base < p.pages && found < asked; base += kPlanThreads) {
    const uint32_t i = base + tid;
    const bool free = i < p.pages && p.owner[i] == 0 && !bit_of(p.bits, i) && !(p.held && p.held[i]);
    unsigned long long total;
    const unsigned long long at = found + block_scan(free ? 1 : 0, warp_sum, &total) - (free ? 1 : 0);
    if (free) p.list[at] = i;
    found += total;
  }
  __syncthreads();
  for (uint32_t r = warp; r < p.rows; r += kPlanThreads / 32) {  // a warp a row
    const uint32_t old = p.len_out[r];
    __syncwarp();
    if (old == CK_NO_PAGE) {
      if (lane == 0) p.len_out[r] = 0;
      continue;
    }
    const uint32_t len = old + p.grow[r], full = old >> p.page_shift, part = old & mask;
    uint32_t last = 0;
    const bool keeps = part && stays(r, old, &last);
    const uint32_t have = full + (keeps ? 1u : 0u), end = (len + mask) >> p.page_shift;
    const unsigned long long first = p.before[r];
    uint32_t* to = p.table_out + (size_t)r * p.stride;
    if (first + (end - have) > found) {
      for (uint32_t i = lane; i < full; i += 32) to[i] = CK_NO_PAGE;
      if (lane == 0) {
        p.status[r] = CK_BUFFER_TOO_SMALL;
        p.len_out[r] = 0;
      }
      continue;
    }
    for (uint32_t i = have + lane; i < end; i += 32) to[i] = p.list[first + (i - have)];
    if (lane == 0) {
      p.len_out[r] = len;
      if (keeps) to[full] = last;
      if (part && !keeps) p.copies[atomicAdd(&n_copies, 1u)] = {last, p.list[first], part, 0};
    }
  }
  __syncthreads();
  if (tid == 0) *p.copied = n_copies;
  if (job.k) copy_pages(job, p.copies, n_copies, warp, kPlanThreads / 32);  // few enough for one block
}

// Packing, first step (a warp a row): checks and marks the row's pages.
__device__ __forceinline__ void compact_mark(const PagesParams& p, uint32_t r, uint32_t lane) {
  const uint32_t len = p.len_in[r];
  uint32_t status = 0;
  if (len > kMaxPositions || len > ((uint64_t)p.stride << p.page_shift)) status = CK_CONTEXT_EXCEEDED;
  const uint32_t n = status ? 0u : (len + (1u << p.page_shift) - 1) >> p.page_shift;
  const uint32_t* from = p.table_in + (size_t)r * p.stride;
  const Kept keeps = kept_pages(len, n, p.sinks, p.window, p.page_shift);
  bool bad = false;
  for (uint32_t i = lane; i < n; i += 32) bad |= keeps(i) && from[i] >= p.pages;
  if (__any_sync(0xffffffffu, bad)) status = CK_INVALID_STATE;
  if (status == 0)
    for (uint32_t i = lane; i < n; i += 32)
      if (keeps(i)) atomicOr(p.bits + (from[i] >> 5), 1u << (from[i] & 31));
  if (lane == 0) p.status[r] = status;
}
__global__ void __launch_bounds__(kTableThreads) k_compact_mark(const PagesParams p) {
  const uint32_t r = blockIdx.x * (kTableThreads / 32) + threadIdx.x / 32;
  if (r < p.rows) compact_mark(p, r, threadIdx.x & 31);
}

// Third step (a warp a row): the row's pages by their new numbers.
__device__ __forceinline__ void compact_table(const PagesParams& p, uint32_t r, uint32_t lane, uint32_t used) {
  const uint32_t n = p.status[r] ? 0u : (p.len_in[r] + (1u << p.page_shift) - 1) >> p.page_shift;
  const Kept keeps = kept_pages(p.len_in[r], n, p.sinks, p.window, p.page_shift);
  for (uint32_t i = lane; i < p.stride; i += 32) {
    uint32_t id = CK_NO_PAGE;
    if (i < n && keeps(i)) {
      id = p.table_in[(size_t)r * p.stride + i];
      if (id >= used) id = p.owner[id];
    }
    p.table_out[(size_t)r * p.stride + i] = id;
  }
}
__global__ void __launch_bounds__(kTableThreads) k_compact_tables(const PagesParams p) {
  const uint32_t r = blockIdx.x * (kTableThreads / 32) + threadIdx.x / 32;
  if (r < p.rows) compact_table(p, r, threadIdx.x & 31, *p.used_out);
}

// Second step (one block): counts the pages in use, pairs those beyond the count with the
// holes below it, and lists the moves; p.owner becomes each moved page's new number.
// ALONE: with the first step before it and the third behind.
template <bool ALONE>
__global__ void __launch_bounds__(kPlanThreads) k_compact_plan(const PagesParams p, const CopyJob job) {
  __shared__ unsigned long long warp_sum[kPlanThreads / 32];
  const uint32_t tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (what follows waits for this grid's end)
  if (ALONE) {
    clear_marks(p);
    for (uint32_t r = tid / 32; r < p.rows; r += kPlanThreads / 32) compact_mark(p, r, tid & 31);
    __syncthreads();
  }
  unsigned long long used = 0;
  const uint32_t words = (p.pages + 31) / 32;
  for (uint32_t base = 0; base < words; base += kPlanThreads) {
    unsigned long long total;
    block_scan(base + tid < words ? __popc(p.bits[base + tid]) : 0, warp_sum, &total);
    used += total;
  }
  unsigned long long holes = 0, movers = 0;
  for (uint32_t base = 0; base < p.pages; base += kPlanThreads) {
    const uint32_t i = base + tid;
    const bool in = i < p.pages && bit_of(p.bits, i);
    const unsigned long long hole = i < used && !in ? 1 : 0, mover = i >= used && in ? 1 : 0;
    unsigned long long total;  // both counts in one scan: pages are below 2^32
    const unsigned long long at = block_scan(hole | mover << 32, warp_sum, &total);
    if (hole) p.list[holes + (uint32_t)at - 1] = i;
    if (mover) p.list2[movers + (at >> 32) - 1] = i;
    holes += (uint32_t)total;
    movers += total >> 32;
  }
  __syncthreads();
  for (uint32_t i = tid; i < movers; i += kPlanThreads) {
    p.owner[p.list2[i]] = p.list[i];
    p.copies[i] = {p.list2[i], p.list[i], 1u << p.page_shift, 0};
  }
  if (tid == 0) {
    *p.copied = (uint32_t)movers;
    *p.used_out = (uint32_t)used;
  }
  if (ALONE) {
    __syncthreads();
    for (uint32_t r = tid / 32; r < p.rows; r += kPlanThreads / 32) compact_table(p, r, tid & 31, (uint32_t)used);
  }
  if (job.k) {  // few enough for one block
    __syncthreads();
    copy_pages(job, p.copies, (uint32_t)movers, tid / 32, kPlanThreads / 32);
  }
}

// Between two passes: sequences give pages back, get pages for their new positions, and the rows
// of the next pass their places.
struct AdvanceParams {
  const uint32_t* len_in;
  const uint32_t* table_in;
  const uint32_t* ask;
  const uint8_t* held;
  uint32_t* len_out;
  uint32_t* table_out;
  uint32_t* start;
  int64_t* slot;
  uint32_t* position;
  uint32_t* status;
  uint32_t seqs, stride, pages, page_shift, rows, sinks, window;
  uint32_t* bits;             // pages that a sequence keeps, but for
  uint32_t* parts;            // those that one goes on in
  uint32_t* apart;            // those held outside the call, where there are any
  uint32_t* list;             // free pages
  // of each sequence the part-filled page that it goes on in, CK_NO_PAGE for none; from the second step on the
  // pages that those before it ask for
  unsigned long long* before;
};

__device__ __forceinline__ uint32_t pages_of(const AdvanceParams& p, uint32_t len) {
  return (len + (1u << p.page_shift) - 1) >> p.page_shift;
}
// Longest sequence a table row holds.
__device__ __forceinline__ uint32_t longest(const AdvanceParams& p) {
  return (uint32_t)min((unsigned long long)p.stride << p.page_shift, (unsigned long long)kMaxPositions);
}

// First step (a warp takes sequence first and every `step`-th behind it, 32 at a time): checks them, takes
// over and marks the pages that their next position or a later one sees.  The part-filled ones that sequences go
// on in have marks of their own, so that a page with both marks is not such a sequence's alone; two of them on a
// page leave both, too.
constexpr uint32_t kEntries = 4;  // of a table row, a lane holds
__device__ __forceinline__ void advance_mark(const AdvanceParams& p, uint32_t* bits, uint32_t* parts, uint32_t first,
                                             uint32_t step, uint32_t lane) {
  for (; first < p.seqs; first += 32 * step) {
    const uint64_t at = first + (uint64_t)lane * step;  // this lane's sequence
    const uint32_t lens = at < p.seqs ? p.len_in[at] : 0, asks = at < p.seqs ? p.ask[at] : 0;
    const uint32_t many = min(32u, (p.seqs - first + step - 1) / step);
    uint32_t my_status = 0, my_part = CK_NO_PAGE;  // this lane's
    for (uint32_t k = 0; k < many; ++k) {
      const uint32_t s = first + k * step, len = __shfl_sync(0xffffffffu, lens, k), ask = __shfl_sync(0xffffffffu, asks, k);
      uint32_t status = 0;
      if (len > longest(p))
        status = CK_INVALID_STATE;
      else if ((unsigned long long)len + ask > longest(p))
        status = CK_CONTEXT_EXCEEDED;
      const uint32_t have = status == CK_INVALID_STATE ? 0 : pages_of(p, len);
      const Kept keeps = kept_pages(len, have, p.sinks, p.window, p.page_shift);
      const uint32_t* from = p.table_in + (size_t)s * p.stride;
      uint32_t* to = p.table_out + (size_t)s * p.stride;
      constexpr uint32_t kStep = 32 * kEntries;
      auto none = [&](uint32_t i0) { return i0 >= have || (i0 >= keeps.early && i0 + kStep <= keeps.late); };  // of a step's entries
      uint32_t id[kEntries];
      auto read = [&](uint32_t i0) {
#pragma unroll
        for (uint32_t j = 0; j < kEntries; ++j) id[j] = keeps(i0 + 32 * j + lane) ? __ldg(from + i0 + 32 * j + lane) : 0;
      };
      uint32_t last = 0xFFFFFFFFu;  // the step that id holds
      bool bad = false;
      for (uint32_t i0 = 0; i0 < have; i0 += kStep) {
        if (none(i0)) continue;
        read(last = i0);
#pragma unroll
        for (uint32_t j = 0; j < kEntries; ++j) bad |= id[j] >= p.pages;
      }
      if (__any_sync(0xffffffffu, bad)) status = CK_INVALID_STATE;
      const bool live = status != CK_INVALID_STATE;
      // the part-filled page that the sequence goes on in
      const uint32_t part_at = status == 0 && ask && (len & ((1u << p.page_shift) - 1)) ? have - 1 : CK_NO_PAGE;
      uint32_t part = 0;
      for (uint32_t i0 = 0; i0 < p.stride; i0 += kStep) {
        const bool empty = !live || none(i0);
        if (!empty && last != i0) read(last = i0);
#pragma unroll
        for (uint32_t j = 0; j < kEntries; ++j) {
          const uint32_t i = i0 + 32 * j + lane;
          const bool kept = !empty && keeps(i);
          if (i < p.stride) to[i] = kept ? id[j] : CK_NO_PAGE;
          if (i == part_at) part = id[j];
          if (kept && i != part_at) atomicOr(bits + (id[j] >> 5), 1u << (id[j] & 31));
        }
      }
      part = __shfl_sync(0xffffffffu, part, part_at & 31);
      if (lane == k) {
        my_status = status;
        my_part = part_at == CK_NO_PAGE ? CK_NO_PAGE : part;
      }
    }
    if (at < p.seqs) {
      p.status[at] = my_status;
      p.before[at] = my_part;
      const uint32_t bit = 1u << (my_part & 31);
      if (my_part != CK_NO_PAGE && (atomicOr(parts + (my_part >> 5), bit) & bit)) atomicOr(bits + (my_part >> 5), bit);
    }
  }
}
// and the pages held outside the call (in words of their own: a sequence may go on in one that is not handed out), of
// which those shared with a sequence there are marked as well: a warp takes the `first`-th eight words of 32 and
// every `step`-th eight behind.
__device__ __forceinline__ void advance_held(const AdvanceParams& p, uint32_t* bits, uint32_t first, uint32_t step, uint32_t lane) {
  const uint32_t words = (p.pages + 31) / 32;
  for (uint32_t w0 = 8 * first; w0 < words; w0 += 8 * step) {
    uint8_t held[8];
    uint32_t mine = 0, shared = 0;  // lane j's words
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) held[j] = (w0 + j) * 32 + lane < p.pages ? __ldg(p.held + (w0 + j) * 32 + lane) : 0;
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) {
      const uint32_t word = __ballot_sync(0xffffffffu, held[j] != 0);
      const uint32_t theirs = __ballot_sync(0xffffffffu, held[j] & CK_PAGE_SHARED);
      if (lane == j) {
        mine = word;
        shared = theirs;
      }
    }
    if (lane < 8 && w0 + lane < words) p.apart[w0 + lane] = mine;
    if (shared) atomicOr(bits + w0 + lane, shared);
  }
}

// Before the second step (one block): the sequences that would go on in a page with both marks are refused.
__device__ __forceinline__ void advance_refuse(const AdvanceParams& p) {
  for (uint32_t s = threadIdx.x; s < p.seqs; s += kPlanThreads) {
    const uint32_t part = (uint32_t)p.before[s];
    if (part != CK_NO_PAGE && bit_of(p.bits, part)) p.status[s] = CK_INVALID_ARGUMENT;
  }
  __syncthreads();
}

// Second step (one block): the free pages in ascending order, as many as are asked for, which
// sequences are served, and where their rows start.  A thread takes sequences that follow one another, so
// that there are three sums over the block.
__device__ __forceinline__ void advance_plan(const AdvanceParams& p, unsigned long long* warp_sum) {
  const uint32_t tid = threadIdx.x, words = (p.pages + 31) / 32;
  const uint32_t each = (p.seqs + kPlanThreads - 1) / kPlanThreads, s0 = min(p.seqs, tid * each), s1 = min(p.seqs, s0 + each);
  auto need_of = [&](uint32_t s, uint32_t ask) {
    const uint32_t len = p.len_in[s];
    return pages_of(p, len + ask) - pages_of(p, len);
  };
  unsigned long long need = 0, ask = 0, asked, total;
  for (uint32_t s = s0; s < s1; ++s) {
    const uint32_t rows = p.status[s] == 0 ? p.ask[s] : 0;
    p.before[s] = need;
    need += rows ? need_of(s, rows) : 0;
    ask += rows;
  }
  const unsigned long long need_before = block_scan(need, warp_sum, &asked) - need;
  unsigned long long found = 0;
  for (uint32_t base = 0; base < words && found < asked; base += 4 * kPlanThreads) {
    uint32_t free[4], count = 0;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      const uint32_t w = base + 4 * tid + j;
      free[j] = w < words ? ~(p.bits[w] | p.parts[w] | (p.held ? p.apart[w] : 0)) : 0;
      if (w == words - 1 && (p.pages & 31)) free[j] &= (1u << (p.pages & 31)) - 1;
      count += __popc(free[j]);
    }
    unsigned long long at = found + block_scan(count, warp_sum, &total) - count;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      for (; free[j] && at < asked; free[j] &= free[j] - 1) p.list[at++] = (base + 4 * tid + j) * 32 + __ffs((int)free[j]) - 1;
    found += total;
  }
  unsigned long long ask_before = block_scan(ask, warp_sum, &total) - ask;
  uint32_t granted = 0;
  for (uint32_t s = s0; s < s1; ++s) {
    if (p.status[s] != 0) continue;
    const uint32_t rows = p.ask[s], pages = need_of(s, rows);
    const unsigned long long before = need_before + p.before[s];
    p.before[s] = before;
    ask_before += rows;
    if ((pages == 0 || before + pages <= found) && (rows == 0 || ask_before <= p.rows))
      granted += rows;
    else
      p.status[s] = CK_BUFFER_TOO_SMALL;
  }
  uint32_t start = (uint32_t)block_scan(granted, warp_sum, &total) - granted;
  for (uint32_t s = s0; s < s1; ++s) {
    p.start[s] = start;
    start += p.status[s] == 0 ? p.ask[s] : 0;
  }
  if (tid == 0) p.start[p.seqs] = (uint32_t)total;
}

// Third step (as the first): their new pages and their rows; and the rows behind the last.
__device__ __forceinline__ void advance_fill(const AdvanceParams& p, uint32_t first, uint32_t step, uint32_t lane) {
  const uint32_t mask = (1u << p.page_shift) - 1;
  for (; first < p.seqs; first += 32 * step) {
    const uint64_t at = first + (uint64_t)lane * step;  // this lane's sequence
    const bool there = at < p.seqs;
    const uint32_t status = there ? p.status[at] : CK_INVALID_STATE, lens = there ? p.len_in[at] : 0;
    const uint32_t wants = there ? p.ask[at] : 0, asks = status == 0 ? wants : 0, starts = there ? p.start[at] : 0;
    const unsigned long long befores = there ? p.before[at] : 0;
    // (the page that the first new position goes on in)
    const uint32_t parts = there && status != CK_INVALID_STATE && (lens & mask) ? p.table_out[at * p.stride + (lens >> p.page_shift)] : 0;
    if (there) p.len_out[at] = status == CK_INVALID_STATE ? 0 : lens + asks;
    // a few new positions a lane by itself, more by the warp together
    auto rows = [&](uint64_t s, uint32_t len, uint32_t ask, uint32_t start, uint32_t part, unsigned long long before,
                    uint32_t j0, uint32_t dj) {
      const uint32_t have = pages_of(p, len), need = pages_of(p, len + ask) - have;
      const uint32_t* fresh = p.list + (need ? before : 0);
      uint32_t* table = p.table_out + s * p.stride;
#pragma unroll 1
      for (uint32_t i = j0; i < need; i += dj) table[have + i] = fresh[i];
#pragma unroll 1
      for (uint32_t j = j0; j < ask; j += dj) {
        const uint32_t pos = len + j, i = pos >> p.page_shift, id = i < have ? part : fresh[i - have];
        p.slot[start + j] = ((int64_t)id << p.page_shift) + (pos & mask);
        p.position[start + j] = pos;
      }
    };
    constexpr uint32_t kFew = 4;
    if (asks && asks <= kFew) rows(at, lens, asks, starts, parts, befores, 0, 1);
    for (uint32_t left = __ballot_sync(0xffffffffu, asks > kFew); left; left &= left - 1) {
      const uint32_t k = __ffs((int)left) - 1;
      rows(first + (uint64_t)k * step, __shfl_sync(0xffffffffu, lens, k), __shfl_sync(0xffffffffu, asks, k),
           __shfl_sync(0xffffffffu, starts, k), __shfl_sync(0xffffffffu, parts, k), __shfl_sync(0xffffffffu, befores, k), lane, 32);
    }
  }
}
__device__ __forceinline__ void advance_rest(const AdvanceParams& p, uint32_t at, uint32_t step) {
  for (uint32_t r = p.start[p.seqs] + at; r < p.rows; r += step) {
    p.slot[r] = -1;
    p.position[r] = CK_NO_PAGE;
  }
}

__global__ void __launch_bounds__(kTableThreads) k_advance_mark(const AdvanceParams p) {
  const uint32_t warps = gridDim.x * (kTableThreads / 32), lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * (kTableThreads / 32) + __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  advance_mark(p, p.bits, p.parts, w, warps, lane);
  if (p.held) advance_held(p, p.bits, w, warps, lane);
}
__global__ void __launch_bounds__(kPlanThreads) k_advance_plan(const AdvanceParams p) {
  __shared__ unsigned long long warp_sum[kPlanThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  advance_refuse(p);
  advance_plan(p, warp_sum);
}
__global__ void __launch_bounds__(kTableThreads) k_advance_fill(const AdvanceParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  advance_fill(p, blockIdx.x * (kTableThreads / 32) + __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), gridDim.x * (kTableThreads / 32), threadIdx.x & 31);
  advance_rest(p, blockIdx.x * kTableThreads + threadIdx.x, gridDim.x * kTableThreads);
}

// All of it in one launch, by a cluster of blocks or one: the steps are separated by the cluster's barriers
// (which order what its blocks write to global memory), the second is the first block's.  Every block marks
// pages in its own shared memory (131,000 atomics on L2 from eight SMs take 17 us).  The chain of loads and
// sums bounds it: 5 us for 4 sequences, 14 for 64 with 512 table entries each, 25 for 2,048 with 128, of which the
// marks for parts take 0.3, 1 and 3 (waiting for what every entry's atomic returns took 5).
constexpr uint32_t kAdvanceBlocks = 8;
__global__ void __launch_bounds__(kPlanThreads) k_advance(const AdvanceParams p, uint32_t blocks) {
  __shared__ unsigned long long warp_sum[kPlanThreads / 32];
  extern __shared__ __align__(16) uint32_t marks[];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warps = blocks * (kPlanThreads / 32), words = (p.pages + 31) / 32;
  const uint32_t w = blockIdx.x * (kPlanThreads / 32) + __shfl_sync(0xffffffffu, tid / 32, 0);
  uint32_t* parts = marks + words;
  __shared__ uint32_t refusals;  // the first block's: some page has both marks
  if (tid == 0) refusals = 0;
  auto sync = [&] {
    if (blocks > 1)
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
      __syncthreads();
  };
  for (uint32_t i = tid; i < 2 * words; i += kPlanThreads) marks[i] = 0;
  __syncthreads();
  advance_mark(p, marks, parts, w, warps, lane);
  if (p.held) advance_held(p, marks, w, warps, lane);
  sync();
  const uint32_t share = (words + blocks - 1) / blocks, end = min(words, (blockIdx.x + 1) * share);
  for (uint32_t i = blockIdx.x * share + tid; i < end; i += kPlanThreads) {
    uint32_t word = marks[i], part = parts[i], others[kAdvanceBlocks], other_parts[kAdvanceBlocks];
#pragma unroll
    for (uint32_t k = 1; k < kAdvanceBlocks; ++k) {  // (all asked for at once)
      others[k] = other_parts[k] = 0;
      if (k < blocks) {
        uint32_t at = (uint32_t)__cvta_generic_to_shared(marks + i);
        asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"((blockIdx.x + k) % blocks));
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(others[k]) : "r"(at) : "memory");
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other_parts[k]) : "r"(at + 4 * words) : "memory");
      }
    }
#pragma unroll
    for (uint32_t k = 1; k < kAdvanceBlocks; ++k) {
      word |= others[k] | (part & other_parts[k]);
      part |= other_parts[k];
    }
    p.bits[i] = word;
    p.parts[i] = part;
    if (word & part) {
      uint32_t at = (uint32_t)__cvta_generic_to_shared(&refusals);
      asm("mapa.shared::cluster.u32 %0, %0, 0;" : "+r"(at));
      asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(at) : "memory");
    }
  }
  sync();  // (and no block leaves while another reads its marks)
  if (blockIdx.x == 0) {
    if (refusals) advance_refuse(p);
    advance_plan(p, warp_sum);
  }
  sync();
  advance_fill(p, w, warps, lane);
  advance_rest(p, blockIdx.x * kPlanThreads + tid, blocks * kPlanThreads);
}

int pages_args(const ck_paged_cache* cache, uint32_t rows, uint32_t stride, void* work, size_t work_len,
               PagesLayout* w) {
  if (!pools_ok(cache) || !work || !aligned_to(work, 256)) return CK_INVALID_ARGUMENT;
  if (rows < 1 || rows > 65536 || stride < 1 || stride > (1u << 17)) return CK_INVALID_ARGUMENT;
  *w = pages_layout(cache->pages, rows);
  return work_len < w->size ? CK_BUFFER_TOO_SMALL : CK_OK;
}

CopyJob copy_job(const ck_paged_cache* c) {
  return {c->dev_k, c->dev_v, c->layers * c->kv_heads, log2_of(c->page), c->head_dim};
}

int run_copies(const ck_paged_cache* c, const PagesParams& p, cudaStream_t s) {
  DeviceFacts f;
  CKP_CUDA(device_facts(&f));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(f.sms * 8);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  CKP_CUDA(cudaLaunchKernelEx(&cfg, k_copy_pages, copy_job(c), static_cast<const Copy*>(p.copies),
                              static_cast<const uint32_t*>(p.copied)));
  return CK_OK;
}

// The copies too, where they move at most 256 KB: of a page a row (a fork) or of as many as lie
// outside the packed range (packing, at most half the pool).
bool copies_alone(const ck_paged_cache* c, uint64_t pages) {
  return 8 * pages * c->layers * c->kv_heads * c->page * c->head_dim <= 256 * 1024;
}

// One block does the table work of a call this small (a row is a warp's, 32 at a time, and a
// thread clears every 1,024th page); larger ones spread it over the GPU.
bool table_work_alone(uint32_t rows, uint32_t stride, uint32_t pages) {
  return (uint64_t)rows * ((stride + 31) / 32) <= 1024 && pages <= 65536;
}

// One cluster does all of a step of up to 2 MB of tables and as many pages as two marks each in shared memory
// allow.  That goes by the time of a call, which the host bounds: 30 us against 35 by a memset and three kernels.  On
// the device, where a captured step is paid, it is 5 against 10 for 4 sequences, 14 and 13 for 64 with 512
// entries each, 16 and 14 for 512 with 256, but 25 and 15 for 2,048 with 128.  A row is a warp's in either:
// one of 131,072 entries takes 590 and 550.
constexpr uint32_t kAdvancePages = 7u << 17;
bool advance_alone(uint32_t seqs, uint32_t stride, uint32_t pages) {
  return (uint64_t)seqs * stride <= (1u << 19) && pages <= kAdvancePages;
}

PagesParams pages_params(const ck_paged_cache* c, const ck_window* window, const PagesLayout& w, void* work) {
  uint8_t* b = static_cast<uint8_t*>(work);
  PagesParams p = {};
  p.pages = c->pages;
  p.page_shift = log2_of(c->page);
  p.sinks = window ? window->sinks : 0;
  p.window = window ? window->window : 0xFFFFFFFFu;
  p.owner = reinterpret_cast<uint32_t*>(b + w.owner);
  p.bits = reinterpret_cast<uint32_t*>(b + w.bits);
  p.copied = reinterpret_cast<uint32_t*>(b + w.counters);
  p.list = reinterpret_cast<uint32_t*>(b + w.list);
  p.list2 = reinterpret_cast<uint32_t*>(b + w.list2);
  p.before = reinterpret_cast<unsigned long long*>(b + w.before);
  p.copies = reinterpret_cast<Copy*>(b + w.copies);
  return p;
}

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" {

int ck_paged_store(const ck_paged_cache* cache, uint32_t layer, const ck_paged_batch* batch,
                   const int64_t* dev_q, size_t q_stride, const int64_t* dev_k, size_t k_stride,
                   const int64_t* dev_v, size_t v_stride, uint32_t heads, const int32_t* dev_rope,
                   uint32_t rope_rows, uint32_t rot, int half, int64_t* dev_q_out, void* stream) {
  if (!pools_ok(cache) || !batch_ok(batch) || layer >= cache->layers) return CK_INVALID_ARGUMENT;
  if (!dev_q || !dev_k || !dev_v || !dev_q_out || heads < 1 || heads > 65536) return CK_INVALID_ARGUMENT;
  if (!aligned_to(dev_q, 16) || !aligned_to(dev_k, 16) || !aligned_to(dev_v, 16) || !aligned_to(dev_q_out, 16))
    return CK_INVALID_ARGUMENT;
  const uint64_t q_dim = (uint64_t)heads * cache->head_dim, kv_dim = (uint64_t)cache->kv_heads * cache->head_dim;
  if (q_stride < q_dim || k_stride < kv_dim || v_stride < kv_dim || (q_stride | k_stride | v_stride) & 1)
    return CK_INVALID_ARGUMENT;
  if ((q_stride | k_stride | v_stride) >> 40) return CK_INVALID_ARGUMENT;
  if (rot > cache->head_dim || rot % 4 || (rot && (!dev_rope || !aligned_to(dev_rope, 16) || rope_rows < 1)))
    return CK_INVALID_ARGUMENT;
  const uint64_t last = batch->rows - 1, out_bytes = 8 * batch->rows * q_dim;
  if (overlaps(dev_q_out, out_bytes, dev_q, 8 * (last * q_stride + q_dim)) ||
      overlaps(dev_q_out, out_bytes, dev_k, 8 * (last * k_stride + kv_dim)) ||
      overlaps(dev_q_out, out_bytes, dev_v, 8 * (last * v_stride + kv_dim)) ||
      overlaps(dev_q_out, out_bytes, dev_rope, 4ull * rope_rows * rot) || on_batch(dev_q_out, out_bytes, *cache, *batch))
    return CK_INVALID_ARGUMENT;
  StoreParams p = {};
  p.pool = pool_view(*cache, layer);
  p.batch = batch_view(*batch);
  p.q = dev_q;
  p.k = dev_k;
  p.v = dev_v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.heads = heads;
  p.rope = dev_rope;
  p.rope_rows = rope_rows;
  p.rot = rot;
  p.half = half ? 1u : 0u;
  p.q_out = dev_q_out;
  DeviceFacts f;
  CKP_CUDA(device_facts(&f));
  const uint32_t units = (heads + 2 * cache->kv_heads) * (cache->head_dim / 4);
  const dim3 grid(batch->rows, batch->rows >= 4u * f.sms ? 1 : (units + kStoreThreads - 1) / kStoreThreads);
  k_paged_store<<<grid, kStoreThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  CKP_CUDA(cudaGetLastError());
  return CK_OK;
}

int ck_pages_work(const ck_paged_cache* cache, uint32_t rows, uint32_t stride, size_t* out) {
  if (!out || !cache_ok(cache) || rows < 1 || rows > 65536 || stride < 1 || stride > (1u << 17))
    return CK_INVALID_ARGUMENT;
  *out = pages_layout(cache->pages, rows).size;
  return CK_OK;
}

int ck_pages_window_fork(const ck_paged_cache* cache, uint32_t rows_in, const uint32_t* dev_len_in,
                         const uint32_t* dev_table_in, uint32_t rows, const uint32_t* dev_parent,
                         const uint32_t* dev_grow, uint32_t stride, const ck_window* window, const uint8_t* dev_held,
                         uint32_t* dev_len_out, uint32_t* dev_table_out, uint32_t* dev_status, void* dev_work,
                         size_t work_len, void* stream) {
  PagesLayout w;
  if (const int rc = pages_args(cache, rows, stride, dev_work, work_len, &w)) return rc;
  if (rows_in < 1 || rows_in > 65536 || !dev_len_in || !dev_table_in || !dev_parent || !dev_grow || !dev_len_out ||
      !dev_table_out || !dev_status || (window && window->window == 0))
    return CK_INVALID_ARGUMENT;
  const void* in[] = {dev_len_in, dev_table_in, dev_parent, dev_grow, dev_held};
  const uint64_t in_bytes[] = {4ull * rows_in, 4ull * rows_in * stride, 4ull * rows, 4ull * rows,
                               dev_held ? cache->pages : 0ull};
  const void* out[] = {dev_len_out, dev_table_out, dev_status, dev_work};
  const uint64_t out_bytes[] = {4ull * rows, 4ull * rows * stride, 4ull * rows, work_len};
  for (int o = 0; o < 4; ++o) {
    if (!aligned_to(out[o], 4) || on_pools(out[o], out_bytes[o], *cache)) return CK_INVALID_ARGUMENT;
    for (int i = 0; i < 5; ++i) {
      if (i < 4 && !aligned_to(in[i], 4)) return CK_INVALID_ARGUMENT;
      if (overlaps(out[o], out_bytes[o], in[i], in_bytes[i])) return CK_INVALID_ARGUMENT;
    }
    for (int i = 0; i < o; ++i)
      if (overlaps(out[o], out_bytes[o], out[i], out_bytes[i])) return CK_INVALID_ARGUMENT;
  }
  PagesParams p = pages_params(cache, window, w, dev_work);
  p.len_in = dev_len_in;
  p.table_in = dev_table_in;
  p.parent = dev_parent;
  p.grow = dev_grow;
  p.held = dev_held;
  p.len_out = dev_len_out;
  p.table_out = dev_table_out;
  p.status = dev_status;
  p.rows_in = rows_in;
  p.rows = rows;
  p.stride = stride;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (table_work_alone(rows, stride, cache->pages)) {
    const bool all = copies_alone(cache, rows);
    k_fork_plan<true><<<1, kPlanThreads, 0, s>>>(p, all ? copy_job(cache) : CopyJob{});
    if (all) {
      CKP_CUDA(cudaGetLastError());
      return CK_OK;
    }
  } else {
    CKP_CUDA(cudaMemsetAsync(dev_work, 0, w.zero, s));
    constexpr uint32_t per = kTableThreads / 32;
    k_fork_mark<<<(rows + per - 1) / per, kTableThreads, 0, s>>>(p);
    k_fork_plan<false><<<1, kPlanThreads, 0, s>>>(p, CopyJob{});
  }
  CKP_CUDA(cudaGetLastError());
  return run_copies(cache, p, s);
}

int ck_pages_fork(const ck_paged_cache* cache, uint32_t rows_in, const uint32_t* dev_len_in,
                  const uint32_t* dev_table_in, uint32_t rows, const uint32_t* dev_parent,
                  const uint32_t* dev_grow, uint32_t stride, const uint8_t* dev_held,
                  uint32_t* dev_len_out, uint32_t* dev_table_out, uint32_t* dev_status, void* dev_work,
                  size_t work_len, void* stream) {
  return ck_pages_window_fork(cache, rows_in, dev_len_in, dev_table_in, rows, dev_parent, dev_grow, stride, nullptr,
                              dev_held, dev_len_out, dev_table_out, dev_status, dev_work, work_len, stream);
}

int ck_pages_window_compact(const ck_paged_cache* cache, uint32_t rows, const uint32_t* dev_len,
                            const uint32_t* dev_table_in, uint32_t stride, const ck_window* window,
                            uint32_t* dev_table_out, uint32_t* dev_used, uint32_t* dev_status, void* dev_work,
                            size_t work_len, void* stream) {
  PagesLayout w;
  if (const int rc = pages_args(cache, rows, stride, dev_work, work_len, &w)) return rc;
  if (!dev_len || !dev_table_in || !dev_table_out || !dev_used || !dev_status || (window && window->window == 0))
    return CK_INVALID_ARGUMENT;
  const void* in[] = {dev_len, dev_table_in};
  const uint64_t in_bytes[] = {4ull * rows, 4ull * rows * stride};
  const void* out[] = {dev_used, dev_table_out, dev_status, dev_work};
  const uint64_t out_bytes[] = {4, 4ull * rows * stride, 4ull * rows, work_len};
  for (int o = 0; o < 4; ++o) {
    if (!aligned_to(out[o], 4) || on_pools(out[o], out_bytes[o], *cache)) return CK_INVALID_ARGUMENT;
    for (int i = 0; i < 2; ++i)
      if (!aligned_to(in[i], 4) || overlaps(out[o], out_bytes[o], in[i], in_bytes[i])) return CK_INVALID_ARGUMENT;
    for (int i = 0; i < o; ++i)
      if (overlaps(out[o], out_bytes[o], out[i], out_bytes[i])) return CK_INVALID_ARGUMENT;
  }
  PagesParams p = pages_params(cache, window, w, dev_work);
  p.len_in = dev_len;
  p.table_in = dev_table_in;
  p.table_out = dev_table_out;
  p.status = dev_status;
  p.used_out = dev_used;
  p.rows = rows;
  p.stride = stride;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (table_work_alone(rows, stride, cache->pages)) {
    const bool all = copies_alone(cache, cache->pages / 2);
    k_compact_plan<true><<<1, kPlanThreads, 0, s>>>(p, all ? copy_job(cache) : CopyJob{});
    if (all) {
      CKP_CUDA(cudaGetLastError());
      return CK_OK;
    }
  } else {
    CKP_CUDA(cudaMemsetAsync(dev_work, 0, w.zero, s));
    constexpr uint32_t per = kTableThreads / 32;
    k_compact_mark<<<(rows + per - 1) / per, kTableThreads, 0, s>>>(p);
    k_compact_plan<false><<<1, kPlanThreads, 0, s>>>(p, CopyJob{});
    k_compact_tables<<<(rows + per - 1) / per, kTableThreads, 0, s>>>(p);
  }
  CKP_CUDA(cudaGetLastError());
  return run_copies(cache, p, s);
}

int ck_pages_compact(const ck_paged_cache* cache, uint32_t rows, const uint32_t* dev_len,
                     const uint32_t* dev_table_in, uint32_t stride, uint32_t* dev_table_out,
                     uint32_t* dev_used, uint32_t* dev_status, void* dev_work, size_t work_len,
                     void* stream) {
  return ck_pages_window_compact(cache, rows, dev_len, dev_table_in, stride, nullptr, dev_table_out, dev_used, dev_status,
                                 dev_work, work_len, stream);
}

int ck_pages_advance(const ck_paged_cache* cache, uint32_t seqs, const uint32_t* dev_len_in,
                     const uint32_t* dev_table_in, const uint32_t* dev_new, uint32_t stride, const ck_window* window,
                     const uint8_t* dev_held, uint32_t rows, uint32_t* dev_len_out, uint32_t* dev_table_out,
                     uint32_t* dev_start, int64_t* dev_slot, uint32_t* dev_position, uint32_t* dev_status,
                     void* dev_work, size_t work_len, void* stream) {
  PagesLayout w;
  if (const int rc = pages_args(cache, seqs, stride, dev_work, work_len, &w)) return rc;
  if (rows < 1 || rows > (1u << 20) || !dev_len_in || !dev_table_in || !dev_new || !dev_len_out || !dev_table_out ||
      !dev_start || !dev_slot || !dev_position || !dev_status || (window && window->window == 0))
    return CK_INVALID_ARGUMENT;
  const void* in[] = {dev_len_in, dev_table_in, dev_new, dev_held};
  const uint64_t in_bytes[] = {4ull * seqs, 4ull * seqs * stride, 4ull * seqs, dev_held ? cache->pages : 0ull};
  const void* out[] = {dev_slot, dev_len_out, dev_table_out, dev_start, dev_position, dev_status, dev_work};
  const uint64_t out_bytes[] = {8ull * rows, 4ull * seqs, 4ull * seqs * stride, 4ull * (seqs + 1), 4ull * rows,
                                4ull * seqs, work_len};
  for (int o = 0; o < 7; ++o) {
    if (!aligned_to(out[o], o ? 4 : 8) || on_pools(out[o], out_bytes[o], *cache)) return CK_INVALID_ARGUMENT;
    for (int i = 0; i < 4; ++i)
      if ((i < 3 && !aligned_to(in[i], 4)) || overlaps(out[o], out_bytes[o], in[i], in_bytes[i]))
        return CK_INVALID_ARGUMENT;
    for (int i = 0; i < o; ++i)
      if (overlaps(out[o], out_bytes[o], out[i], out_bytes[i])) return CK_INVALID_ARGUMENT;
  }
  AdvanceParams p = {};
  p.len_in = dev_len_in;
  p.table_in = dev_table_in;
  p.ask = dev_new;
  p.held = dev_held;
  p.len_out = dev_len_out;
  p.table_out = dev_table_out;
  p.start = dev_start;
  p.slot = dev_slot;
  p.position = dev_position;
  p.status = dev_status;
  p.seqs = seqs;
  p.stride = stride;
  p.pages = cache->pages;
  p.page_shift = log2_of(cache->page);
  p.rows = rows;
  p.sinks = window ? window->sinks : 0;
  p.window = window ? window->window : 0xFFFFFFFFu;
  uint8_t* b = static_cast<uint8_t*>(dev_work);
  const uint32_t words = (p.pages + 31) / 32;
  p.bits = reinterpret_cast<uint32_t*>(b + w.bits);
  p.parts = p.bits - words;  // (at the end of the owners, which a step doesn't use, as it doesn't the second list)
  p.apart = reinterpret_cast<uint32_t*>(b + w.list2);
  p.list = reinterpret_cast<uint32_t*>(b + w.list);
  p.before = reinterpret_cast<unsigned long long*>(b + w.before);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (advance_alone(seqs, stride, cache->pages)) {
    const uint32_t blocks = seqs <= kPlanThreads / 32 && cache->pages <= 65536 ? 1 : kAdvanceBlocks;  // (a warp a sequence)
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kPlanThreads);
    DeviceFacts f;
    CKP_CUDA(device_facts(&f));
    static std::atomic<bool> ready[64];
    if (!ready[f.dev].load(std::memory_order_relaxed)) {
      CKP_CUDA(cudaFuncSetAttribute(k_advance, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kAdvancePages / 8));
      ready[f.dev].store(true, std::memory_order_relaxed);
    }
    cfg.dynamicSmemBytes = 8 * words;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    CKP_CUDA(cudaLaunchKernelEx(&cfg, k_advance, p, blocks));
    return CK_OK;
  }
  CKP_CUDA(cudaMemsetAsync(p.parts, 0, 8ull * words, s));  // and the bits behind it
  constexpr uint32_t per = kTableThreads / 32;
  const uint32_t blocks = (seqs + per - 1) / per;
  k_advance_mark<<<blocks, kTableThreads, 0, s>>>(p);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  CKP_CUDA(cudaLaunchKernelEx(&cfg, k_advance_plan, p));
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kTableThreads);
  CKP_CUDA(cudaLaunchKernelEx(&cfg, k_advance_fill, p));
  CKP_CUDA(cudaGetLastError());
  return CK_OK;
}

}  // extern "C"

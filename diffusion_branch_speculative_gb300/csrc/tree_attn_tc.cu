// Tree attention with many rows a head group on the 5th-generation tensor
// cores.  A unit's piece (tree_sched.cuh) is up to 256 query rows of one
// sequence's key/value head over a run of 128-key blocks of its cache.
//
// Two lanes share the pipeline, each with 128 query rows, a score buffer S and an
// output accumulator O in TMEM: while the softmax of one lane runs, the tensor
// cores work for the other.  A piece of more than 128 rows gives each lane its
// half of the rows and both lanes every block (so a block is read once for 256
// rows); one of at most 128 rows gives both lanes the same rows and alternate
// blocks, merged at the end like split units.
//   S = Q K^T (128 x 128 x HD), softmax with one thread per row, P as bf16 (the
//   tensor cores' operand: each weight off by half a step) back over S in TMEM,
//   O += P V with P read from TMEM.
// Head size 64 leaves P columns of its own, so that S of the next block goes ahead
// of P V.
// P in TMEM keeps it out of shared memory, whose 128 bytes a cycle are what such
// products run short of.  A lane's chain of S, softmax and P V is what bounds
// a block: the products alone take 2050 cycles for both lanes, 2700 beside the
// loads and the softmax's TMEM traffic, the chain 3900.  Measured (us, with the
// merge; floors by 6690 GB/s and 1925 TFLOP/s; 8, 4 and 8 key/value heads):
//   1 sequence of 40000 tokens, 61 rows of 3 heads a group     51.2  (floor 24.6)
//   16 padded sequences of 8192, 33 rows of 7                  63.8  (29.3)
//   32 sequences of 8192, 128 rows of 3                       248 to 260 by the box (120.9)
// The tensor cores are busy 35, 33 and 44 % of the kernel's time; start, first
// loads and merge are some 12 us of each.  No faster, beside 58.7, 65.5 and 246
// before the merge was: two threads a row (640 threads; 67, 72, 271), P handed
// over by halves (60.4, 68.2, 257), all 128 scores of a row in registers (59.9,
// 66.1, 250), the first keys ahead of all other loads (61.5, 70.4, 268: CTAs in
// step ask the memory in bursts), 64 keys a step.
//
// Roles (384 threads of 168 registers, which spill 40 bytes, 84 for head size 64): warp 0 loads keys, warp 1 values, both the queries; warp 2
// issues all products (warp 3 owns the TMEM allocation), warps 4-7 and 8-11 are
// the lanes' softmax.  One issuer, so that a lane's P V and next Q K^T go out in
// one run and the lanes fall into alternation (with an issuer each, both lanes'
// products interleaved, both S came at once and the tensor cores idled through
// both softmaxes: 4700-5000 cycles a block against 3950).  A run of products is
// followed by one commit alone, since a second one waits for the products: tiles
// are released by the softmax (which has seen S) and by the issuer (which has
// seen P V).
// K and V tiles (128 keys) go through a ring each.
// They come by TMA, one box per run of tokens inside a page (page_size's power
// of two, 8 to 64), the boxes issued by a warp's threads side by side; boxes
// past the sequence read zeros, and a block that holds the tree's tokens, or
// ends the sequence, has its values mended before they are handed on.  Which of
// its tokens a row sees is 64 bits a step, found by walking up its ancestors.
#include "tree_sched.cuh"

namespace sf {
namespace {

constexpr int kTcThreads = 384;
constexpr int kAtom = 128 * 128;  // one 128-row x 128-byte swizzle block
constexpr int kOddBufs = 4;       // units whose odd-value notes may be alive at once

struct TcArgs {
  CUtensorMap mapK, mapV;  // {dim, heads, pool tokens}, box {64, 1, box}
  TreeArgs t;
  int box;  // tokens of a box
};

template <int HD>
struct Tc {
  static constexpr int NATOM = HD / 64;
  static constexpr int Q_BYTES = kAtom * NATOM;     // of one lane
  static constexpr int TILE = kAtom * NATOM;        // 128 keys' K or V
  // tiles in flight; a value tile waits longer for its use
  static constexpr int KRING = HD == 128 ? 2 : 5, VRING = HD == 128 ? 3 : 5, RING = KRING + VRING;
  static constexpr int OFF_RING = 2 * Q_BYTES;
  static constexpr int SMEM = OFF_RING + RING * TILE + 1024;  // and the base's alignment
  // TMEM: S of lane x at 128 x, O at COL_O + HD x, P over S's columns from 64 on, or,
  // where O leaves room (APART), in columns of its own: then the next S goes ahead of
  // P V (32 sequences of 8000 tokens, 192 rows: 182 us, not 203)
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_O = 256;
  static constexpr bool APART = HD == 64;
  static constexpr uint32_t col_p(int x) { return APART ? 384 + x * 64 : x * 128 + 64; }
};

// The products and commits of a warp that runs as one, issued by the thread with
// `me` set: with the whole warp converged the descriptors stay in uniform
// registers (a single thread's branch moves each there first: 80 cycles a
// product, above its 64 of execution).
// D[tmem] (+)= A[smem] * B[smem]^T
SF_DEV void warp_mma(bool me, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(me))
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T: A's row r in TMEM lane r, two bf16 of
// consecutive k a column.
SF_DEV void warp_mma_ta(bool me, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(me))
      : "memory");
}
SF_DEV void warp_commit(bool me, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar),
      "r"(static_cast<uint32_t>(me))
      : "memory");
}
// Store 16 consecutive 32-bit columns of this thread's TMEM lane.
SF_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// The maximum of three in one instruction.
SF_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Which of the 128 tokens e0, e0 + 1, ... behind the cached ones (negative: still
// cached) node i sees, as bits: the cached ones, itself and its ancestors.  For
// a node that is no padding row.  par: the sequence's parents, null: a chain.
SF_DEV void sees_window(const int32_t* par, int i, int e0, uint32_t* status, uint64_t (&bits)[2]) {
  // tokens [0, n) of the window
  auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; };
  if (!par) {
    bits[0] = below(i + 1 - e0);
    bits[1] = below(i + 1 - e0 - 64);
    return;
  }
  bits[0] = below(-e0);
  bits[1] = below(-e0 - 64);
  int a = i, up = par[i];
  while (a >= e0) {
    const int at = a - e0;
    if (at < 64)
      bits[0] |= 1ull << at;
    else if (at < 128)
      bits[1] |= 1ull << (at - 64);
    if (up == -1) break;
    int above = SPECFOLD_TREE_PAD;
    if (up >= 0 && up < a) above = par[up];
    if (above == SPECFOLD_TREE_PAD) {  // not a parent
      atomicOr(status, SPECFOLD_DEV_BAD_PARENT);
      break;
    }
    a = up;
    up = above;
  }
}

// A tile's queries into the lanes' places, by THREADS threads (thread tid); rows
// past the tile's become zeros.  Returns with this thread's part visible to the
// tensor cores.
template <int HD, int THREADS>
SF_DEV void gather_queries(const TreeArgs& p, const TreeWalk& w, uint8_t* smem, int tid) {
  constexpr int RSTEP = THREADS / (HD / 8);  // rows of one step; a row's node and head follow by steps
  const int g = p.g, rows = tree_tile_rows(p, w), most = rows > 128 ? 256 : 128;
  const int c = tid % (HD / 8), dn = RSTEP / g, dh = RSTEP % g, m = tree_m0(p, w) + tid / (HD / 8);
  int hd = m % g;
  const long long d_node = p.q_rs - g * p.q_hs, d_step = dn * p.q_rs + dh * p.q_hs;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (w.q.row0 + m / g) * p.q_rs +
                             (w.head * g + hd) * p.q_hs + c * 8;
  const uint32_t q0 = smem_u32(smem) + (c >> 3) * kAtom;
#pragma unroll 4
  for (int r = tid / (HD / 8); r < most; r += RSTEP) {
    const bool there = r < rows;
    cp_async16(q0 + (r >> 7) * Tc<HD>::Q_BYTES + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4),
               there ? src : static_cast<const __nv_bfloat16*>(p.q), there ? 16u : 0u);
    src += d_step;
    hd += dh;
    if (hd >= g) {
      hd -= g;
      src += d_node;
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  fence_proxy_async_smem();
}

template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1) tree_attn_tc_kernel(const __grid_constant__ TcArgs ta) {
  using C = Tc<HD>;
  const TreeArgs& p = ta.t;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bars[2 * C::RING + 11];
  __shared__ uint32_t tmem_slot_s;
  __shared__ volatile int abort_s;
  __shared__ float2 xch[128];
  // nodes whose values are not all finite, by unit (see the loaders)
  __shared__ uint32_t odd[kOddBufs][SPECFOLD_MAX_TREE / 32];
  uint64_t* full = bars;                // [RING]: the keys' tiles, then the values'
  uint64_t* empty = bars + C::RING;     // [RING]: a key tile's two arrivals (the lanes'), a value tile's one
  uint64_t* q_full = bars + 2 * C::RING;
  uint64_t* q_empty = q_full + 1;       // both lanes' S products of a unit are done: Q may be replaced
  uint64_t* s_full = q_full + 2;        // [lane]: one completion per block of the lane
  uint64_t* p_full = q_full + 4;        // [lane]
  uint64_t* o_full = q_full + 6;        // [lane]
  uint64_t* o_empty = q_full + 8;       // the softmax warps have read a unit's outputs
  uint64_t* landed = q_full + 9;        // a value tile that is mended before it is handed on
  uint64_t* drain = q_full + 10;
  volatile int* abort_flag = &abort_s;

  // lane 0's copy: the compiler then knows that a warp's role is one
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(q_full), 2);  // the two loading warps, or the lanes' softmax
    mbar_init(smem_u32(q_empty), 2);
    for (int i = 0; i < C::RING; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), i < C::KRING ? 2 : 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&s_full[x]), 1);
      mbar_init(smem_u32(&p_full[x]), 4);  // one arrival a warp: 128 would queue at the barrier's word
      mbar_init(smem_u32(&o_full[x]), 1);
    }
    mbar_init(smem_u32(o_empty), 8);
    mbar_init(smem_u32(landed), 1);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&ta.mapK);
    prefetch_tmap(&ta.mapV);
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(&tmem_slot_s), C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  TreeWalk w;
  unsigned per;
  const bool work = tree_locate(p, w, per);
  if (threadIdx.x == 0) tree_describe(p, w, work, per);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot_s;
  if (!work) {
    if (warp == 3) tmem_dealloc(tmem, C::TMEM_COLS);
    return;
  }
  const int g = p.g;

  // Every role walks the same pieces in the same order; j counts them, it the
  // blocks (tiles of each ring).  The lanes use K of block t + lead after V of
  // block t: lead 1, or 2 where they take alternate blocks.
  if (warp < 2) {
    // ------------------------------------------------------------ loaders --
    const bool is_v = warp == 1;
    const CUtensorMap* map = is_v ? &ta.mapV : &ta.mapK;
    int it = 0, j = 0, issued = -1, fixes = 0;
    bool ok = true;
    const int boxes = kTreeTcKeys / ta.box, ps = p.cache.page_size;
    const int pool = p.cache.num_pages * ps;
    const int box = lane & 15, atom = lane >> 4;  // what this thread issues of a tile
    const bool issues = box < boxes && atom < C::NATOM;
    for (; w.n > 0 && ok; w.next(p), ++j) {
      const int h = w.head, rows = tree_tile_rows(p, w), ctx = w.q.ctx, len = ctx + w.q.n;
      const int nt = w.n, lead = rows > 128 ? 1 : 2;
      // queries, by both warps: the previous unit's S products must be done with
      // their place (the first unit's come from the softmax warps, idle then)
      auto load_queries = [&]() {
        if (j == 0) return true;
        const bool free = lane == 0 ? mbar_wait(smem_u32(q_empty), (j - 1) & 1, abort_flag, p.status, kWaitLimitNs,
                                                kSiteAttnQEmpty)
                                    : true;
        if (!__shfl_sync(0xffffffffu, free, 0)) return false;
        gather_queries<HD, 64>(p, w, smem, threadIdx.x);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(q_full));
        return true;
      };
      const int heads_k = min(lead, nt);
      if (is_v && !load_queries()) {
        ok = false;
        break;
      }
      // this thread's box of the next tile: the table's entry is read a tile
      // ahead of its use and looked at only then
      const unsigned tok0 = static_cast<unsigned>(w.b0) * kTreeTcKeys + box * ta.box;
      int pg = tok0 / static_cast<unsigned>(ps), off = tok0 - pg * ps;
      const int dpg = kTreeTcKeys / ps, doff = kTreeTcKeys - dpg * ps;
      const int32_t* table = p.cache.block_table + w.s * p.cache.table_stride;
      long long left = static_cast<long long>(len) - tok0;  // tokens from the box's first on
      auto entry = [&](int t) {
        return issues && t < nt && left > 0 && pg < p.cache.table_pages ? table[pg] : -1;
      };
      int page = entry(0);
      if (is_v && lane < SPECFOLD_MAX_TREE / 32) odd[j % kOddBufs][lane] = 0u;
      for (int t = 0; t < nt; ++t) {
        if (!is_v && t == heads_k && !load_queries()) {  // behind the first keys' loads
          ok = false;
          break;
        }
        const int i = it + t, turn = i / (is_v ? C::VRING : C::KRING);
        const int st = is_v ? C::KRING + i % C::VRING : i % C::KRING;
        const bool mend = is_v && static_cast<long long>(w.b0 + t + 1) * kTreeTcKeys > ctx;
        const uint32_t fb = smem_u32(mend ? landed : &full[st]);
        if (lane == 0) {
          ok = mbar_wait(smem_u32(&empty[st]), (turn & 1) ^ 1, abort_flag, p.status, kWaitLimitNs,
                         kSiteAttnKvEmpty);
          if (ok) mbar_arrive_expect_tx(fb, C::TILE);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (!mend) issued = i;
        uint8_t* tile = smem + C::OFF_RING + st * C::TILE;
        if (issues) {
          const bool there = page >= 0 && page < p.cache.num_pages;
          if (!there && left > 0) atomicOr(p.status, SPECFOLD_DEV_BAD_PAGE);
          // a box without a page lies wholly past the pool: it reads zeros
          tma_load_3d(smem_u32(tile + atom * kAtom + box * ta.box * 128), map, fb, atom * 64, h,
                      there && left > 0 ? page * ps + off : pool);
        }
        left -= kTreeTcKeys;
        pg += dpg;
        off += doff;
        if (off >= ps) {
          off -= ps;
          ++pg;
        }
        page = entry(t + 1);
        if (mend) {
          // Tokens past the end may hold anything, and a weight of zero does
          // not silence an infinite value or a NaN in a product: values past
          // the end become zeros; such values of the tree's tokens are taken
          // out, noted, and added at the end to the rows that see them.
          const bool there = mbar_wait(smem_u32(landed), fixes & 1, abort_flag, p.status, kWaitLimitNs, kSiteAttnKvFull);
          ++fixes;
          const long long t0 = static_cast<long long>(w.b0 + t) * kTreeTcKeys;
          // rows of the tile: the tree's from r0 on, past the end from r1 on
          const int r0 = t0 >= ctx ? 0 : static_cast<int>(ctx - t0);
          const int r1 = len - t0 >= 128 ? 128 : static_cast<int>(len - t0);
          constexpr int RSTEP = 32 / (HD / 8);
          const int c = lane % (HD / 8), rl = lane / (HD / 8);
          uint8_t* col = tile + (c >> 3) * kAtom;
          auto piece = [&](int r) { return reinterpret_cast<uint4*>(col + r * 128 + (((c & 7) ^ (r & 7)) << 4)); };
          if (there) {
            for (int r = r1 + rl; r < 128; r += RSTEP) *piece(r) = make_uint4(0u, 0u, 0u, 0u);
            // an exponent of ones carries into the place above it
            auto odd_of = [](uint32_t v) { return ((v & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
            for (int rb = r0; rb < r1; rb += 8 * RSTEP) {
              uint4 u[8];  // all read before any is looked at
#pragma unroll
              for (int k = 0; k < 8; ++k) u[k] = *piece(min(rb + rl + k * RSTEP, r1 - 1));
              uint32_t any = 0u;
#pragma unroll
              for (int k = 0; k < 8; ++k) any |= odd_of(u[k].x) | odd_of(u[k].y) | odd_of(u[k].z) | odd_of(u[k].w);
              if (any) {
#pragma unroll 1
                for (int r = rb + rl; r < min(rb + 8 * RSTEP, r1); r += RSTEP) {
                  const uint4 v = *piece(r);
                  uint32_t y[4] = {v.x, v.y, v.z, v.w};
                  if (!(odd_of(v.x) | odd_of(v.y) | odd_of(v.z) | odd_of(v.w))) continue;
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    if ((y[q] & 0x7f80u) == 0x7f80u) y[q] &= 0xffff0000u;
                    if ((y[q] & 0x7f800000u) == 0x7f800000u) y[q] &= 0xffffu;
                  }
                  *piece(r) = make_uint4(y[0], y[1], y[2], y[3]);
                  const int e = static_cast<int>(t0 - ctx) + r;
                  atomicOr(&odd[j % kOddBufs][e >> 5], 1u << (e & 31));
                }
              }
              __syncwarp();
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&full[st]));
        }
      }
      if (ok && !is_v && nt == heads_k) ok = load_queries();
      it += nt;
    }
    if (lane == 0 && *abort_flag) {
      // let the copies already issued land before the CTA exits
      int never = 0;
      if (issued >= 0) {
        const int ring = is_v ? C::VRING : C::KRING;
        mbar_wait(smem_u32(&full[(is_v ? C::KRING : 0) + issued % ring]), (issued / ring) & 1, &never, nullptr, 10000000ull);
      }
      if (fixes > 0) mbar_wait(smem_u32(landed), (fixes - 1) & 1, &never, nullptr, 10000000ull);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax --
    // A row's thread raises its reference maximum m, and rescales O in place,
    // only when the maximum grows by more than 2^8, so weights stay below 2^8.
    // S of a lane's block being there means that P V of its previous one is
    // done (it was waited for), so O may be rescaled; with P apart that wait is here.
    const int x = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    constexpr int OH = HD / 2;
    const uint32_t tS = tmem + lane_off + x * 128;
    const uint32_t tP = tmem + lane_off + C::col_p(x);
    const uint32_t tO = tmem + lane_off + C::COL_O;  // lane 0's; lane 1's HD columns on
    const int pair_bar = 2 + (warp & 3);  // named barrier of the two warps of these rows
    int cnt = 0, j = 0, it = 0;  // blocks of this lane so far
    const bool leader = (warp & 3) == 0 && lane == 0;
    gather_queries<HD, 256>(p, w, smem, threadIdx.x - 128);
    named_bar_sync(1, 256);
    if (leader) mbar_arrive(smem_u32(q_full));
    bool ok = true;
    for (bool first = true; w.n > 0 && ok; first = false, w.next(p), ++j) {
      const int h = w.head, ctx = w.q.ctx, nt = w.n, rows = tree_tile_rows(p, w);
      const bool pair = rows > 128;
      const int r = pair ? x * 128 + row : row;  // row of the tile
      const bool valid = r < rows;
      const int m = valid ? tree_m0(p, w) + r : 0, node = m / g;
      const int32_t* par = p.parent ? p.parent + w.q.row0 : nullptr;
      const bool dead = !valid || (par && par[node] == SPECFOLD_TREE_PAD);  // sees nothing
      float m_ref = -INFINITY, l = 0.f;
      const int t_step = pair ? 1 : 2;
      bool began = false;
      if (leader && !pair && x >= nt) mbar_arrive(smem_u32(q_empty));  // no block of this unit
      for (int t = pair ? 0 : x; t < nt; t += t_step, ++cnt) {
        const int key0 = (w.b0 + t) * kTreeTcKeys;
        const bool allv = key0 + kTreeTcKeys <= ctx;
        uint64_t km[2] = {0ull, 0ull};  // what the row sees of these keys, where not all
        if (!allv && !dead) sees_window(par, node, key0 - ctx, p.status, km);
        // every wait's outcome is made warp-uniform: a lane whose wait ran out
        // takes its whole warp along
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s_full[x]), cnt & 1, abort_flag, p.status, kWaitLimitNs,
                                               kSiteAttnSFull))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (leader) {  // S is there: its keys are done with, and after the last one the queries
          const uint32_t eb = smem_u32(&empty[(it + t) % C::KRING]);
          mbar_arrive(eb);
          if (!pair) mbar_arrive(eb);
          if (t + t_step >= nt) mbar_arrive(smem_u32(q_empty));
        }
        // Two passes of 64 columns: the maximum over the first half, which is
        // read again after the second's weights (128 scores a thread would not
        // fit its registers beside the rest).
        uint32_t sv[2][32];
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto mask = [&](int half) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((km[half] >> (32 * c + e)) & 1u)) sv[c][e] = 0xff800000u;  // -inf
        };
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          tmem_ld32(tS + half * 64, sv[0]);
          tmem_ld32(tS + half * 64 + 32, sv[1]);
          tmem_ld_wait(sv[0]);
          tmem_ld_wait(sv[1]);
          if (!allv) mask(half);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mx4[(e >> 1) & 3] = max3(mx4[(e >> 1) & 3], __uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1]));
        }
        if (C::APART && began &&  // O and P are free once the lane's last P V is done
            !__all_sync(0xffffffffu, mbar_wait(smem_u32(&o_full[x]), (cnt - 1) & 1, abort_flag, p.status, kWaitLimitNs,
                                               kSiteAttnSFree))) {
          ok = false;
          break;
        }
        if (C::APART) tc_fence_after();
        const float mx = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
        const float m_new = fmaxf(m_ref, mx * p.sl2);
        float alpha = 1.f;
        bool rescale = false;
        if (m_ref == -INFINITY) {
          m_ref = m_new;  // nothing accumulated yet (every earlier weight was 0)
        } else if (m_new > m_ref + 8.f) {
          alpha = ex2(m_ref - m_new);
          m_ref = m_new;
          rescale = true;
        }
        l *= alpha;
        if (began && __any_sync(0xffffffffu, rescale)) {
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t q[32];
            tmem_ld32(tO + x * HD + c * 32, q);
            tmem_ld_wait(q);
#pragma unroll
            for (int e = 0; e < 32; ++e) q[e] = __float_as_uint(__uint_as_float(q[e]) * alpha);
            tmem_st32(tO + x * HD + c * 32, q);
          }
        }
        began = true;
        const float base = m_ref == -INFINITY ? 0.f : m_ref;
        const float2 scale2 = make_float2(p.sl2, p.sl2), base2 = make_float2(-base, -base);
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // the second half's weights from the registers into P's upper columns,
        // then the first half's, read again, into its lower ones (over scores
        // that have been used)
        auto weights = [&](int c, int column) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 y = fma2(make_float2(__uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1])), scale2, base2);
            y = make_float2(ex2(y.x), ex2(y.y));
            ls[(e >> 1) & 1] = add2(ls[(e >> 1) & 1], y);
            pk[e / 2] = pack_bf16x2(y.x, y.y);
          }
          tmem_st16(tP + column, pk);
        };
        weights(0, 32);
        tmem_ld32(tS, sv[0]);
        weights(1, 48);
        tmem_ld32(tS + 32, sv[1]);
        tmem_ld_wait(sv[0]);
        tmem_ld_wait(sv[1]);
        if (!allv) mask(0);
        weights(0, 0);
        weights(1, 16);
        l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[x]));
      }
      // this lane's last P V (a lane without blocks has none to wait for)
      const bool oku = ok && (!began || mbar_wait(smem_u32(&o_full[x]), (cnt - 1) & 1, abort_flag, p.status,
                                                  kWaitLimitNs, kSiteAttnEnd));
      // the lanes' meeting: both leave together or neither.  Where they share
      // rows, lane 1 hands its (m, l) to lane 0, which computes the merge's
      // factors and hands lane 1 its pair back; the first barrier also orders
      // lane 0's reads of the previous unit's hand-back before this write.
      const bool whole = w.whole();
      if (x == 1) xch[row] = make_float2(m_ref, l);
      tc_fence_before();
      __syncwarp();
      if (!named_bar_and(pair_bar, 64, oku)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool other = pair || nt > 1;  // lane 1 had blocks
      float a0 = whole ? merge_scale(l) : 1.f, a1 = 0.f, M = m_ref, lrow = l;
      if (!pair) {
        if (x == 0) {
          const float2 o1 = xch[row];
          M = fmaxf(m_ref, o1.x);
          const float w0 = merge_weight(m_ref, M), w1 = other ? merge_weight(o1.x, M) : 0.f;
          lrow = w0 * l + w1 * o1.y;
          const float sc = whole ? merge_scale(lrow) : 1.f;  // a partial stays unnormalised
          a0 = w0 * sc;
          a1 = w1 * sc;
          xch[row] = make_float2(a0, a1);
        }
        named_bar_sync(pair_bar, 64);
        if (x == 1) {
          const float2 f = xch[row];
          a0 = f.x;
          a1 = f.y;
        }
      }
      uint32_t any_odd = 0u;
#pragma unroll
      for (int k = 0; k < SPECFOLD_MAX_TREE / 32; ++k) any_odd |= odd[j % kOddBufs][k];
      const size_t ps = static_cast<size_t>(tree_slot(first)) * p.tile_rows;
      __nv_bfloat16* dst =
          static_cast<__nv_bfloat16*>(p.o) + (w.q.row0 + node) * p.o_rs + (h * g + m % g) * p.o_hs;
      // columns this thread writes: all of its lane's, or half of the shared rows'
      const int c_lo = pair || x == 0 ? 0 : OH / 32, c_hi = pair || x == 1 ? HD / 32 : OH / 32;
#pragma unroll 1
      for (int c = c_lo; c < c_hi; ++c) {
        float o[32];
        {
          uint32_t q[32];
          tmem_ld32(tO + (pair ? x * HD : 0) + c * 32, q);
          tmem_ld_wait(q);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = a0 * __uint_as_float(q[e]);
        }
        if (!pair && other) {
          uint32_t q[32];
          tmem_ld32(tO + HD + c * 32, q);
          tmem_ld_wait(q);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(a1, __uint_as_float(q[e]), o[e]);
        }
        if (any_odd && !dead) {  // rare: infinities and NaN among the tree's values
          for (int i = 0; i <= node; ++i) {
            const int tok = ctx + i;
            if (!(odd[j % kOddBufs][i >> 5] >> (i & 31) & 1u)) continue;
            uint64_t seen[2];
            sees_window(par, node, i, p.status, seen);
            if (!(seen[0] & 1ull)) continue;
            const int at = tree_pool_token(p, w.s, tok);
            if (at < 0) continue;
            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.cache.v) + at * p.cache.v_token_stride +
                                     h * p.cache.v_head_stride + c * 32;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float xv = __bfloat162float(v[e]);
              if (!isfinite(xv)) o[e] += xv;
            }
          }
        }
        if (dead) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (valid && whole) {
#pragma unroll
          for (int q8 = 0; q8 < 4; ++q8)
            reinterpret_cast<uint4*>(dst)[c * 4 + q8] =
                make_uint4(pack_bf16x2(o[8 * q8], o[8 * q8 + 1]), pack_bf16x2(o[8 * q8 + 2], o[8 * q8 + 3]),
                           pack_bf16x2(o[8 * q8 + 4], o[8 * q8 + 5]), pack_bf16x2(o[8 * q8 + 6], o[8 * q8 + 7]));
        } else if (valid) {
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4)  // [quad of columns][row]: a warp's rows side by side
            reinterpret_cast<float4*>(p.part_o + ps * HD)[(c * 8 + q4) * p.tile_rows + r] =
                make_float4(o[4 * q4], o[4 * q4 + 1], o[4 * q4 + 2], o[4 * q4 + 3]);
        }
        __syncwarp();  // the next load of TMEM is the whole warp's
      }
      if (!whole && valid && (pair || x == 0)) {
        p.part_ml[(ps + r) * 2] = dead ? -INFINITY : M;
        p.part_ml[(ps + r) * 2 + 1] = dead ? 0.f : lrow;
      }
      // the accumulators are free for the next unit's first P V products
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(o_empty));
      it += nt;
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- MMA --
    // The whole warp runs this, lane 0 issues; values that all lanes have alike
    // are taken from lane 0 where the compiler could not know it.
    constexpr uint32_t idS = idesc_bf16_f32(128, 128, false);
    constexpr uint32_t idPV = idesc_bf16_f32(128, HD, true);
    const bool me = lane == 0;
    int it = 0, j = 0;
    int cnt0 = 0, cnt1 = 0;  // the lanes' P V products so far
    bool ok = true;
    auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    auto wait = [&](uint64_t* bar, int parity, int site) {
      ok = __all_sync(0xffffffffu,
                      ok && mbar_wait(smem_u32(bar), parity & 1, abort_flag, p.status, kWaitLimitNs, site));
      return ok;
    };
    // two waits, both asked at once (each takes a good hundred cycles)
    auto wait2 = [&](uint64_t* a, int pa, int sa, uint64_t* b, int pb, int sb) {
      const bool ra = mbar_try_wait(smem_u32(a), pa & 1), rb = mbar_try_wait(smem_u32(b), pb & 1);
      if (__all_sync(0xffffffffu, ra && rb && ok)) return true;
      return wait(a, pa, sa) && wait(b, pb, sb);
    };
    auto v_at = [&](int i) { return C::KRING + i % C::VRING; };
    auto k_there = [&](int i) { return wait(&full[i % C::KRING], i / C::KRING, kSiteAttnKvFull); };
    const uint32_t base = uniform(smem_u32(smem)), tm = uniform(tmem);
    // S = Q K^T of lane x with the keys of block i, once the lane's last P V
    // has read P from S's place
    auto issue_s = [&](int x, int i, uint32_t aQ) {
      tc_fence_after();
      const uint32_t aK = base + C::OFF_RING + (i % C::KRING) * C::TILE;
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        warp_mma(me, tm + x * 128, sdesc_sw128(aQ + (kk >> 2) * kAtom + (kk & 3) * 32, 16, 1024),
                 sdesc_sw128(aK + (kk >> 2) * kAtom + (kk & 3) * 32, 16, 1024), idS, kk > 0 ? 1u : 0u);
      warp_commit(me, smem_u32(&s_full[x]));
    };
    for (; uniform(w.n > 0) && ok; w.next(p), ++j) {
      const int nt = uniform(w.n);
      const bool pair = uniform(tree_tile_rows(p, w) > 128);
      const int lead = pair ? 1 : 2;
      const uint32_t aQ1 = base + (pair ? C::Q_BYTES : 0);
      if (!wait(q_full, j, kSiteAttnQFull)) break;
      for (int x = 0; x < 2 && (pair || x < nt); ++x) {  // the lanes' first S
        const int i = it + (pair ? 0 : x), c = x ? cnt1 : cnt0;
        if (!k_there(i) || (c > 0 && !wait(&o_full[x], c - 1, kSiteAttnSFree))) break;
        issue_s(x, i, x ? aQ1 : base);
      }
      // P V of lane x's next block with the values of block i; first: the unit's
      // first, which overwrites O (read by then, see its wait)
      auto issue_pv = [&](int x, int i, bool first) {
        if (first && j > 0 && !wait(o_empty, j - 1, kSiteAttnOEmpty)) return;
        tc_fence_after();
        const uint32_t aV = base + C::OFF_RING + v_at(i) * C::TILE;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          warp_mma_ta(me, tm + C::COL_O + x * HD, tm + C::col_p(x) + kk * 8, sdesc_sw128(aV + kk * 2048, kAtom, 1024),
                      idPV, (!first || kk > 0) ? 1u : 0u);
        warp_commit(me, smem_u32(&o_full[x]));
      };
      for (int t = 0; t < nt && ok; ++t) {
        const int iv = it + t, ik = it + t + lead;
        const bool more = t + lead < nt;
        uint64_t *vf = &full[v_at(iv)], *kf = &full[ik % C::KRING], *ve = &empty[v_at(iv)];
        if constexpr (C::APART) {  // a lane's next S once P is there, then its P V
          for (int x = pair ? 0 : t & 1; x < (pair ? 2 : (t & 1) + 1) && ok; ++x) {
            const int c = x ? cnt1 : cnt0;
            if (!wait2(vf, iv / C::VRING, kSiteAttnKvFull, &p_full[x], c, kSiteAttnPFull)) break;
            if (more) {
              if (!k_there(ik)) break;
              issue_s(x, ik, x ? aQ1 : base);
            }
            issue_pv(x, iv, pair ? t == 0 : t < 2);
            if (!ok) break;
            if (!pair || x == 1) warp_commit(me, smem_u32(ve));
            x ? ++cnt1 : ++cnt0;
          }
          continue;
        }
        // lane 0, or the only lane of this block
        const int x = pair ? 0 : t & 1;
        if (!wait2(vf, iv / C::VRING, kSiteAttnKvFull, &p_full[x], x ? cnt1 : cnt0, kSiteAttnPFull)) break;
        issue_pv(x, iv, pair ? t == 0 : t < 2);
        x ? ++cnt1 : ++cnt0;
        if (more && wait2(kf, ik / C::KRING, kSiteAttnKvFull, &o_full[x], (x ? cnt1 : cnt0) - 1, kSiteAttnSFree)) {
          if (!pair && me) mbar_arrive(smem_u32(ve));  // the values are done with
          issue_s(x, ik, x ? aQ1 : base);
        }
        if (pair && ok) {  // lane 1
          if (!wait(&p_full[1], cnt1, kSiteAttnPFull)) break;
          issue_pv(1, iv, t == 0);
          ++cnt1;
          if (more && wait(&o_full[1], cnt1 - 1, kSiteAttnSFree)) {
            if (me) mbar_arrive(smem_u32(ve));
            issue_s(1, ik, aQ1);
          }
        }
        if (!more) warp_commit(me, smem_u32(ve));
      }
      it += nt;
    }
    warp_commit(me, smem_u32(drain));
    int never = 0;
    mbar_wait(smem_u32(drain), 0, &never, nullptr, 10000000ull);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int HD>
int tc_go(const TreeArgs& a, int grid, cudaStream_t st) {
  using C = Tc<HD>;
  TcArgs ta;
  ta.t = a;
  const specfold_paged_cache& c = a.cache;
  ta.box = c.page_size % 64 == 0 ? 64 : c.page_size % 32 == 0 ? 32 : c.page_size % 16 == 0 ? 16 : 8;
  const uint64_t tokens = static_cast<uint64_t>(c.num_pages) * c.page_size;
  // L2 fetches a row: with 256 bytes for rows of 128 the other half would be another
  // head's (32 sequences of 8000 tokens, 64 rows, head size 64: 105 us, not 140; the
  // same 104 where a head's rows lie side by side)
  constexpr int kRow = HD * 2;
  if (const int rc = make_map_3d(&ta.mapK, c.k, HD, a.n_kv, tokens, c.k_head_stride, c.k_token_stride, ta.box, kRow))
    return rc;
  if (const int rc = make_map_3d(&ta.mapV, c.v, HD, a.n_kv, tokens, c.v_head_stride, c.v_token_stride, ta.box, kRow))
    return rc;
  if (const int rc = smem_limit_once(tree_attn_tc_kernel<HD>, C::SMEM)) return rc;
  launch_k(tree_attn_tc_kernel<HD>, dim3(grid), dim3(kTcThreads), C::SMEM, st, ta);
  count_launch();
  return check_launch();
}

}  // namespace

int launch_tree_tc(const TreeArgs& a, int hd, int grid, cudaStream_t st) {
  return hd == 128 ? tc_go<128>(a, grid, st) : tc_go<64>(a, grid, st);
}

}  // namespace sf

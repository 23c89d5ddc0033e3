// Attention of drafted rows over a paged cache and their tree
// (specfold_tree_attention): the fp32 kernel, the bf16 kernel for few rows a head
// group, and the merge of split units.  tree_sched.cuh has the decomposition,
// tree_attn_tc.cu the bf16 kernel for many rows.
#include "tree_sched.cuh"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

namespace sf {
namespace {

constexpr int kThreads = 128;  // 4 warps, each with its own chunks of keys
constexpr int kWarps = kThreads / 32;
constexpr int kFewKeys = 64;   // keys of a block of these kernels: a chunk or two of each warp's
constexpr int kSmBudget = 160; // SMs the workspace is sized for (>= one GB300)

SF_DEV float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
SF_DEV void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
SF_DEV void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// The four warps' (o [RT][HD], {m, l} [RT]), `stride` bytes apart, into the
// output of the current piece's rows, or into its partial slot.
template <typename T, int HD, int RT>
SF_DEV void merge_warps(const TreeArgs& p, const TreeWalk& w, bool first, const uint8_t* smem, int stride) {
  const int h = w.head, m0 = tree_m0(p, w), rows = tree_tile_rows(p, w);
  const bool whole = w.whole();
  const size_t ps = static_cast<size_t>(tree_slot(first)) * p.tile_rows;
  const float* mw = reinterpret_cast<const float*>(smem);
  const int ws = stride / 4;
  for (int i = threadIdx.x; i < rows * (HD / 4); i += kThreads) {
    const int r = i / (HD / 4), d = (i % (HD / 4)) * 4;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, mw[k * ws + RT * HD + 2 * r]);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float wk = merge_weight(mw[k * ws + RT * HD + 2 * r], M);
      const float4 v = load4(mw + k * ws + r * HD + d);
      L = fmaf(wk, mw[k * ws + RT * HD + 2 * r + 1], L);
      a.x = fmaf(wk, v.x, a.x);
      a.y = fmaf(wk, v.y, a.y);
      a.z = fmaf(wk, v.z, a.z);
      a.w = fmaf(wk, v.w, a.w);
    }
    if (whole) {
      const int m = m0 + r;
      const float sc = merge_scale(L);
      if (L == 0.f) a = make_float4(0.f, 0.f, 0.f, 0.f);
      store4(static_cast<T*>(p.o) + (w.q.row0 + m / p.g) * p.o_rs + (h * p.g + m % p.g) * p.o_hs + d,
             make_float4(a.x * sc, a.y * sc, a.z * sc, a.w * sc));
    } else {
      store4(p.part_o + (ps + r) * HD + d, a);
      if (d == 0) {
        p.part_ml[(ps + r) * 2] = M;
        p.part_ml[(ps + r) * 2 + 1] = L;
      }
    }
  }
}

// ------------------------------------------------------ fp32: CUDA cores --
// Tiles of RT rows (row m = node m / g, head m % g of the group).  Every warp
// streams its own 4 KB chunks of keys through a private ring of asynchronous
// copies, with its own running maximum and sum, so the loop has no block-wide
// barrier; the four warps merge once per piece.
//   scores: lane = (key, 32 of the dimensions), the row's query broadcast
//           from shared memory, a key's lanes joined by shuffles;
//   output: lane = dimensions, the probabilities broadcast.
// A chunk's 16-byte pieces are stored with their index xored with the row's low
// three bits, so that eight rows read at one place never share a bank.  A piece
// of at most RT / 2 rows does no other rows' arithmetic.
// Few rows are bound by the memory, more by the reads of shared memory (nine of
// 16 bytes for 32 multiply-adds a lane).  Measured (16 sequences of 4000 tokens,
// 4 key/value heads; copy peak 6690 GB/s): head size 128, 2 rows 0.26 GB in
// 51.4 us (5100 GB/s; all eight rows' arithmetic 75.9; with one CTA an SM for
// 16-key chunks 90.8), 16 rows in two tiles 144.5 us; head size 64 31.2 and
// 75.3 us (two CTAs an SM instead of three: 50.8 and 90.7 with eight rows each).
template <int HD>
struct Simt {
  using T = float;
  static constexpr int RT = 8;
  static constexpr int CH = 1024 / HD;              // keys of a warp's step: 4 KB, and as much of values
  static constexpr int STAGES = 2;
  static constexpr int ROW = HD * sizeof(T);        // bytes of a key
  static constexpr int CPR = ROW / 16;              // 16-byte pieces of a key
  static constexpr int STAGE = 2 * CH * ROW;        // keys, then values
  static constexpr int RING = STAGES * STAGE;       // of one warp
  static constexpr int MERGE = RT * (HD + 2) * 4;   // of one warp, over its ring
  static constexpr int OFF_Q = kWarps * (RING > MERGE ? RING : MERGE);
  static constexpr int OFF_P = OFF_Q + RT * HD * 4;
  static constexpr int SMEM = OFF_P + kWarps * CH * RT * 4;
  static constexpr int CTAS = 3;  // per SM: 68 to 71 KB each (168 registers; head size 128 spills 8 bytes)
};

template <int HD>
__global__ void __launch_bounds__(kThreads, Simt<HD>::CTAS) tree_attn_simt_kernel(const __grid_constant__ TreeArgs p) {
  using C = Simt<HD>;
  using T = float;
  constexpr int RT = C::RT, CH = C::CH, DPL = HD / 32;  // dimensions of the output a lane holds
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int16_t s_parent[SPECFOLD_MAX_TREE];
  __shared__ uint32_t s_sees[RT][SPECFOLD_MAX_TREE / 32];  // a tile row's ancestors and itself
  __shared__ int s_dead[RT];                               // padding rows
  pdl_wait();
  pdl_trigger();
  TreeWalk w;
  unsigned per;
  const bool work = tree_locate(p, w, per);
  if (threadIdx.x == 0) tree_describe(p, w, work, per);
  if (!work) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * (C::RING > C::MERGE ? C::RING : C::MERGE);
  float* s_q = reinterpret_cast<float*>(smem + C::OFF_Q);
  float* s_p = reinterpret_cast<float*>(smem + C::OFF_P) + warp * CH * RT;
  const T* qp = static_cast<const T*>(p.q);

  for (bool first = true; w.n > 0; first = false, w.next(p)) {
    const int h = w.head, m0 = tree_m0(p, w), rows = tree_tile_rows(p, w);
    const int len = w.q.ctx + w.q.n, key_lo = w.b0 * p.kb;
    const int key_hi = min(static_cast<long long>(len), static_cast<long long>(w.b0 + w.n) * p.kb);
    __syncthreads();  // the previous piece's shared memory is free
    for (int i = threadIdx.x; i < RT * (HD / 4); i += kThreads) {
      const int r = i / (HD / 4), d = (i % (HD / 4)) * 4, m = m0 + r;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) v = load4(qp + (w.q.row0 + m / p.g) * p.q_rs + (h * p.g + m % p.g) * p.q_hs + d);
      store4(s_q + r * HD + d, v);
    }
    for (int i = threadIdx.x; i < w.q.n; i += kThreads) {
      int a = p.parent ? p.parent[w.q.row0 + i] : i - 1;
      if (a < SPECFOLD_TREE_PAD || a >= i || (a >= 0 && p.parent && p.parent[w.q.row0 + a] == SPECFOLD_TREE_PAD)) {
        a = -1;
        atomicOr(p.status, SPECFOLD_DEV_BAD_PARENT);
      }
      s_parent[i] = static_cast<int16_t>(a);
    }
    __syncthreads();
    if (threadIdx.x < RT) {
      const int r = threadIdx.x;
      for (int k = 0; k < SPECFOLD_MAX_TREE / 32; ++k) s_sees[r][k] = 0u;
      const int i = r < rows ? (m0 + r) / p.g : 0;
      s_dead[r] = r >= rows || s_parent[i] == SPECFOLD_TREE_PAD;
      if (!s_dead[r])
        for (int a = i; a >= 0; a = s_parent[a]) s_sees[r][a >> 5] |= 1u << (a & 31);
    }
    __syncthreads();

    // this warp's chunks: key_lo + CH * (warp + 4 i)
    const int chunks = (key_hi - key_lo + CH - 1) / CH;
    const int mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
    auto key_of = [&](int i) { return key_lo + CH * (warp + kWarps * i); };
    auto slot_of = [&](int i) {  // lanes 0..CH-1: pool tokens of chunk i's keys
      const int tok = key_of(i) + (lane & (CH - 1));
      return i < mine && tok < key_hi ? tree_pool_token(p, w.s, tok) : -1;
    };
    auto load = [&](int i, int slot) {
      if (i < mine) {
        uint8_t* st = ring + (i % C::STAGES) * C::STAGE;
#pragma unroll
        for (int it = 0; it < 2 * CH * C::CPR / 32; ++it) {
          const int idx = it * 32 + lane;
          const int c = idx % C::CPR, key = (idx / C::CPR) % CH, is_v = idx / (C::CPR * CH);
          const int tk = __shfl_sync(0xffffffffu, slot, key);
          const T* src = is_v ? static_cast<const T*>(p.cache.v) + tk * p.cache.v_token_stride + h * p.cache.v_head_stride
                              : static_cast<const T*>(p.cache.k) + tk * p.cache.k_token_stride + h * p.cache.k_head_stride;
          if (tk < 0) src = static_cast<const T*>(p.cache.k);  // any valid address: nothing is read
          cp_async16(smem_u32(st + is_v * CH * C::ROW + key * C::ROW + ((c ^ (key & 7)) << 4)),
                     reinterpret_cast<const uint8_t*>(src) + (tk < 0 ? 0 : c * 16), tk < 0 ? 0u : 16u);
        }
      }
      cp_async_commit();
    };
    auto at = [](const uint8_t* rows_, int key, int d) {  // address of dimension d of a stored key
      const int b = d * static_cast<int>(sizeof(T));
      return reinterpret_cast<const T*>(rows_ + key * C::ROW + (((b >> 4) ^ (key & 7)) << 4) + (b & 15));
    };

    float mx[RT], l[RT], acc[RT][DPL];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      mx[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int d = 0; d < DPL; ++d) acc[r][d] = 0.f;
    }
    int slot = slot_of(0);
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) {
      load(i, slot);
      slot = slot_of(i + 1);
    }
    auto stream = [&](auto nr) {
      constexpr int NR = decltype(nr)::value;  // rows worked on
      for (int i = 0; i < mine; ++i) {
        load(i + C::STAGES - 1, slot);
        slot = slot_of(i + C::STAGES);
        cp_async_wait<C::STAGES - 1>();
        __syncwarp();
        const uint8_t* sk = ring + (i % C::STAGES) * C::STAGE;
        const uint8_t* sv = sk + CH * C::ROW;
        const int key = lane & (CH - 1), part = lane / CH;
        float s[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) s[r] = 0.f;
#pragma unroll
        for (int d = 0; d < 32; d += 4) {
          const float4 k4 = load4(at(sk, key, part * 32 + d));
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float4 q4 = load4(s_q + r * HD + part * 32 + d);
            s[r] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[r]))));
          }
        }
        const int tok = key_of(i) + key, e = tok - w.q.ctx;
        const bool tail = key_of(i) + CH > w.q.ctx;  // holds tokens that not every row sees
        float pr[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int o = CH; o < 32; o <<= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
          bool see = !s_dead[r];
          if (tail) see = see && tok < key_hi && (e < 0 || (s_sees[r][(e >> 5) & 7] >> (e & 31) & 1u));
          s[r] = see ? s[r] * p.sl2 : -INFINITY;
          float m = s[r];
#pragma unroll
          for (int o = CH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          m = fmaxf(m, mx[r]);
          const float base = m == -INFINITY ? 0.f : m;
          const float alpha = mx[r] == m ? 1.f : ex2(mx[r] - base);
          pr[r] = see ? ex2(s[r] - base) : 0.f;
          mx[r] = m;
          l[r] = l[r] * alpha + pr[r];
          if (alpha != 1.f) {
#pragma unroll
            for (int d = 0; d < DPL; ++d) acc[r][d] *= alpha;
          }
        }
        if (part == 0) {
#pragma unroll
          for (int r = 0; r < NR; r += 4) store4(s_p + key * RT + r, make_float4(pr[r], pr[r + 1], pr[r + 2], pr[r + 3]));
        }
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < CH; ++k) {
          float v[DPL];
          const T* vp = at(sv, k, lane * DPL);
#pragma unroll
          for (int d = 0; d < DPL; ++d) v[d] = static_cast<float>(vp[d]);
#pragma unroll
          for (int r0 = 0; r0 < NR; r0 += 4) {
            const float4 p4 = load4(s_p + k * RT + r0);
            const float pk[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              // a token the row does not see adds nothing, whatever its value
              if (!tail || pk[r] != 0.f) {
#pragma unroll
                for (int d = 0; d < DPL; ++d) acc[r0 + r][d] = fmaf(pk[r], v[d], acc[r0 + r][d]);
              }
            }
          }
        }
        __syncwarp();  // the stage and the probabilities may be overwritten
      }
    };
    if (rows <= RT / 2)
      stream(std::integral_constant<int, RT / 2>{});
    else
      stream(std::integral_constant<int, RT>{});
    cp_async_wait<0>();
    __syncwarp();

    // the warps' merge: each writes (o, m, l) over its own ring
    float* mo = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float ls = l[r];
#pragma unroll
      for (int o = CH / 2; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
#pragma unroll
      for (int d = 0; d < DPL; ++d) mo[r * HD + lane * DPL + d] = acc[r][d];
      if (lane == 0) {
        mo[RT * HD + 2 * r] = mx[r];
        mo[RT * HD + 2 * r + 1] = ls;
      }
    }
    __syncthreads();
    merge_warps<T, HD, RT>(p, w, first, smem, C::RING > C::MERGE ? C::RING : C::MERGE);
  }
}

// ---------------------------------------------------- few rows, bf16: mma --
// Up to RT = 16 MT rows of a head group (a whole sequence's nodes times the
// group; MT 2 for head size 64 alone): decoding and small trees.  Such a unit
// does at most 32 operations a byte of cache, so the memory bounds it and
// warp-level matrix instructions, whose rows fit, are enough; what counts is
// bytes in flight and no barrier between them.  So, as above, each of the four warps streams its own 4 KB
// chunks of keys through a private ring of asynchronous copies:
//   S [rows x chunk] = Q K^T, keys as the B operand straight from their rows;
//   O [rows x HD] += P V, P from S's registers (rounded to bf16, the tensor
//   cores' operand: off by half a step of each weight), V's rows transposed
//   by the load.
// 64 KB in flight an SM would cover the latency at full bandwidth; two CTAs of
// 96 KB keep it covered while one of them merges.  Measured (32 sequences of 8000
// tokens, 8 key/value heads, 4 rows; copy peak 6690 GB/s): head size 128
// 1.05 GB in 162 us (6470 GB/s; one CTA an SM 233), head size 64 0.52 GB in
// 90 us (5820 GB/s; chunks of 16 keys with two or four CTAs 107 and 117).
// 8 sequences of 500 tokens: 10.9 and 8.6 us, the latency of the two launches.
template <int HD, int MT>
struct Few {
  static constexpr int RT = 16 * MT;
  static constexpr int CH = 2048 / HD;  // keys of a warp's step: 4 KB, and as much of values
  static constexpr int STAGES = 3;
  static constexpr int ROW = HD * 2;
  static constexpr int CPR = ROW / 16;
  static constexpr int STAGE = 2 * CH * ROW;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int MERGE = RT * (HD + 2) * 4;
  static_assert(MERGE <= RING, "the merge goes over the ring");
  static constexpr int OFF_Q = kWarps * RING;
  static constexpr int SMEM = OFF_Q + RT * ROW;
  static constexpr int CTAS = 2;  // per SM
  static constexpr bool Q_IN_REGS = MT == 1;      // two row tiles' queries would not fit beside their outputs
};

SF_DEV bool bf16_not_finite(uint32_t x) {  // either half
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}

template <int HD, int MT>
__global__ void __launch_bounds__(kThreads, Few<HD, MT>::CTAS) tree_attn_few_kernel(const __grid_constant__ TreeArgs p) {
  using C = Few<HD, MT>;
  using T = __nv_bfloat16;
  constexpr int RT = C::RT, KS = HD / 16, CH = C::CH, KH = CH / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_wait();
  pdl_trigger();
  TreeWalk w;
  unsigned per;
  const bool work = tree_locate(p, w, per);
  if (threadIdx.x == 0) tree_describe(p, w, work, per);
  if (!work) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * C::RING;
  uint8_t* s_q = smem + C::OFF_Q;
  // a stored row's 16-byte piece c lies at c ^ (row & 7): the eight rows of a
  // matrix load then never share a bank
  auto q_addr = [&](int mt, int ks) {
    const int r = mt * 16 + (lane & 15);
    return smem_u32(s_q + r * C::ROW + (((ks * 2 + (lane >> 4)) ^ (r & 7)) << 4));
  };

  for (bool first = true; w.n > 0; first = false, w.next(p)) {
    const int h = w.head, rows = w.q.n * p.g;
    const int len = w.q.ctx + w.q.n, key_lo = w.b0 * p.kb;
    const int key_hi = min(static_cast<long long>(len), static_cast<long long>(w.b0 + w.n) * p.kb);
    __syncthreads();  // the previous piece's shared memory is free

    // this warp's chunks: key_lo + CH * (warp + 4 i)
    const int chunks = (key_hi - key_lo + CH - 1) / CH;
    const int mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
    auto key_of = [&](int i) { return key_lo + CH * (warp + kWarps * i); };
    auto slot_of = [&](int i) {  // lanes 0..CH-1: pool tokens of chunk i's keys
      const int tok = key_of(i) + (lane & (CH - 1));
      return i < mine && tok < key_hi ? tree_pool_token(p, w.s, tok) : -1;
    };
    const T* kbase = static_cast<const T*>(p.cache.k) + h * p.cache.k_head_stride;
    const T* vbase = static_cast<const T*>(p.cache.v) + h * p.cache.v_head_stride;
    auto load = [&](int i, int slot) {
      if (i < mine) {
        const uint32_t st = smem_u32(ring + (i % C::STAGES) * C::STAGE);
        constexpr int KEYS = 32 / C::CPR;  // keys of one step of the warp's lanes
        const int c = lane % C::CPR;
#pragma unroll
        for (int it = 0; it < CH / KEYS; ++it) {
          const int key = it * KEYS + lane / C::CPR;
          const int tk = __shfl_sync(0xffffffffu, slot, key);
          const uint32_t n = tk < 0 ? 0u : 16u, at = st + key * C::ROW + ((c ^ (key & 7)) << 4);
          const long long tz = tk < 0 ? 0 : tk;  // any valid address when nothing is read
          cp_async16(at, kbase + tz * p.cache.k_token_stride + c * 8, n);
          cp_async16(at + CH * C::ROW, vbase + tz * p.cache.v_token_stride + c * 8, n);
        }
      }
      cp_async_commit();
    };
    int slot = slot_of(0);
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) {
      load(i, slot);
      slot = slot_of(i + 1);
    }

    // queries: row m = node m / g, head m % g of the group
    for (int i = threadIdx.x; i < RT * C::CPR; i += kThreads) {
      const int r = i / C::CPR, c = i % C::CPR;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows)
        v = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (w.q.row0 + r / p.g) * p.q_rs +
                                            (h * p.g + r % p.g) * p.q_hs + c * 8);
      *reinterpret_cast<uint4*>(s_q + r * C::ROW + ((c ^ (r & 7)) << 4)) = v;
    }
    // ancestors: lane i has node i's, by doubling its jump towards the root
    uint32_t sees = 0u;
    {
      const bool live = lane < w.q.n;
      const int raw = !live ? SPECFOLD_TREE_PAD : p.parent ? p.parent[w.q.row0 + lane] : lane - 1;
      int jump = raw;
      const int up = __shfl_sync(0xffffffffu, raw, raw >= 0 ? raw & 31 : 0);
      if (live && raw != SPECFOLD_TREE_PAD &&
          (raw < -1 || raw >= lane || (raw >= 0 && up == SPECFOLD_TREE_PAD))) {
        jump = -1;
        if (warp == 0) atomicOr(p.status, SPECFOLD_DEV_BAD_PARENT);
      }
      if (raw != SPECFOLD_TREE_PAD) sees = 1u << lane;
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        const int from = max(jump, 0);
        const uint32_t more = __shfl_sync(0xffffffffu, sees, from);
        const int next = __shfl_sync(0xffffffffu, jump, from);
        if (jump >= 0) {
          sees |= more;
          jump = next;
        }
      }
    }
    uint32_t vis[MT][2];  // what this thread's rows see of the tree; 0: nothing at all
#pragma unroll
    for (int q = 0; q < 2 * MT; ++q) {
      const int r = (q >> 1) * 16 + (q & 1) * 8 + (lane >> 2);
      const uint32_t v = __shfl_sync(0xffffffffu, sees, r < rows ? r / p.g : 0);
      vis[q >> 1][q & 1] = r < rows ? v : 0u;
    }
    __syncthreads();
    uint32_t qf[KS][4];
    if constexpr (C::Q_IN_REGS) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) ldsm4(q_addr(0, ks), qf[ks]);
    }

    float mx[MT][2], l[MT][2], o[MT][HD / 8][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      mx[mt][0] = mx[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < HD / 8; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
    }
    for (int i = 0; i < mine; ++i) {
      load(i + C::STAGES - 1, slot);
      slot = slot_of(i + C::STAGES);
      cp_async_wait<C::STAGES - 1>();
      __syncwarp();
      uint8_t* stg = ring + (i % C::STAGES) * C::STAGE;
      uint8_t* sv = stg + CH * C::ROW;
      float s[MT][2 * KH][4] = {};
      {
        const int key = (lane & 7) + ((lane >> 4) << 3);
        const uint32_t base = smem_u32(stg + key * C::ROW);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t a[MT][4];
          if constexpr (!C::Q_IN_REGS) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) ldsm4(q_addr(mt, ks), a[mt]);
          }
#pragma unroll
          for (int kh = 0; kh < KH; ++kh) {
            uint32_t b[4];
            ldsm4(base + kh * 16 * C::ROW + (((ks * 2 + ((lane >> 3) & 1)) ^ (key & 7)) << 4), b);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint32_t(&q)[4] = C::Q_IN_REGS ? qf[ks] : a[mt];
              mma16816(s[mt][2 * kh], q, b[0], b[1]);
              mma16816(s[mt][2 * kh + 1], q, b[2], b[3]);
            }
          }
        }
      }
      const int e0 = key_of(i) - w.q.ctx;
      const bool tail = e0 + CH > 0;  // holds tokens that not every row sees
      if (tail) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 8 * KH; ++x) {
            const int e = e0 + (x >> 2) * 8 + (lane & 3) * 2 + (x & 1);
            const bool see = e < 0 || (e < 32 && (vis[mt][(x >> 1) & 1] >> (e & 31) & 1u));
            if (!see) s[mt][x >> 2][x & 3] = -INFINITY;
          }
      }
      uint32_t pf[MT][KH][4];
      bool grew = false;
      float alpha[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          float m = fmaxf(s[mt][0][2 * hr], s[mt][0][2 * hr + 1]);
#pragma unroll
          for (int j = 1; j < 2 * KH; ++j) m = fmaxf(m, fmaxf(s[mt][j][2 * hr], s[mt][j][2 * hr + 1]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          m = fmaxf(m * p.sl2, mx[mt][hr]);
          const float base = m == -INFINITY ? 0.f : m;
          alpha[mt][hr] = mx[mt][hr] == m ? 1.f : ex2(mx[mt][hr] - base);
          grew = grew || mx[mt][hr] != m;
          mx[mt][hr] = m;
          l[mt][hr] *= alpha[mt][hr];
#pragma unroll
          for (int kh = 0; kh < KH; ++kh) {
            float pr[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) pr[x] = ex2(fmaf(s[mt][2 * kh + (x >> 1)][2 * hr + (x & 1)], p.sl2, -base));
            l[mt][hr] += (pr[0] + pr[1]) + (pr[2] + pr[3]);
            pf[mt][kh][hr] = pack_bf16x2(pr[0], pr[1]);
            pf[mt][kh][2 + hr] = pack_bf16x2(pr[2], pr[3]);
          }
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < HD / 8; ++j) {
            o[mt][j][0] *= alpha[mt][0];
            o[mt][j][1] *= alpha[mt][0];
            o[mt][j][2] *= alpha[mt][1];
            o[mt][j][3] *= alpha[mt][1];
          }
      }
      if (tail) {
        // a weight of zero does not silence an infinite value or a NaN in a
        // product, so such values of the tree's rows are added by hand to the
        // rows that see them and then taken out
        bool odd = false;
        for (int x = lane; x < CH * C::CPR; x += 32) {
          const uint4 u = *reinterpret_cast<const uint4*>(sv + x * 16);
          odd = odd || bf16_not_finite(u.x) || bf16_not_finite(u.y) || bf16_not_finite(u.z) || bf16_not_finite(u.w);
        }
        if (__any_sync(0xffffffffu, odd)) {
          for (int k = 0; k < CH; ++k) {
            const int e = e0 + k;
#pragma unroll
            for (int j = 0; j < HD / 8; ++j) {
              const uint32_t u = *reinterpret_cast<const uint32_t*>(sv + k * C::ROW + ((j ^ (k & 7)) << 4) + (lane & 3) * 4);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const bool see = e < 0 || (e < 32 && (vis[mt][x >> 1] >> (e & 31) & 1u));
                  const float v = (x & 1) ? bf16hi(u) : bf16lo(u);
                  if (see && !isfinite(v)) o[mt][j][x] += v;
                }
            }
          }
          __syncwarp();
          for (int x = lane; x < CH * C::CPR * 8; x += 32) {
            uint16_t* v = reinterpret_cast<uint16_t*>(sv) + x;
            if ((*v & 0x7f80u) == 0x7f80u) *v = 0;
          }
          __syncwarp();
        }
      }
      {
        const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t base = smem_u32(sv + key * C::ROW);
#pragma unroll
        for (int kh = 0; kh < KH; ++kh)
#pragma unroll
          for (int j = 0; j < HD / 16; ++j) {
            uint32_t b[4];
            ldsm4t(base + kh * 16 * C::ROW + (((j * 2 + (lane >> 4)) ^ (key & 7)) << 4), b);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816(o[mt][2 * j], pf[mt][kh], b[0], b[1]);
              mma16816(o[mt][2 * j + 1], pf[mt][kh], b[2], b[3]);
            }
          }
      }
      __syncwarp();  // the stage may be overwritten
    }
    cp_async_wait<0>();
    __syncwarp();

    float* mo = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const int r = mt * 16 + hr * 8 + (lane >> 2);
        const bool dead = vis[mt][hr] == 0u;
        float ls = l[mt][hr];
        ls += __shfl_xor_sync(0xffffffffu, ls, 1);
        ls += __shfl_xor_sync(0xffffffffu, ls, 2);
#pragma unroll
        for (int j = 0; j < HD / 8; ++j)
          *reinterpret_cast<float2*>(mo + r * HD + j * 8 + (lane & 3) * 2) =
              dead ? make_float2(0.f, 0.f) : make_float2(o[mt][j][2 * hr], o[mt][j][2 * hr + 1]);
        if ((lane & 3) == 0) {
          mo[RT * HD + 2 * r] = dead ? -INFINITY : mx[mt][hr];
          mo[RT * HD + 2 * r + 1] = dead ? 0.f : ls;
        }
      }
    __syncthreads();
    merge_warps<T, HD, RT>(p, w, first, smem, C::RING);
  }
}

// ---------------------------------------------------------------- combine --
// Merges the partials of cut units: block (c, y) has four rows of the unit that
// CTA c's start cuts first.  The partials of one unit lie at its first CTA's slot
// and at the first slots of the CTAs after it; each of the block's warps takes
// every eighth of them, all rows at once, with a running maximum and sum of its
// own, and the warps merge at the end.  One sequence of 40000 tokens (76 partials
// a unit of 7 rows) takes 19.9 us in all, 28.5 with a warp a row that goes through
// its partials alone; 64 sequences of 8000 (2 a unit) 168 us either way.  Eight
// rows a block: 20.9, two 19.6 but 14.5 instead of 12.4 for 8 sequences of 500
// tokens and 32 rows; four warps a block 23.4.  Merging by the last CTA of a unit
// to arrive, without a launch: 26.5 and 184, and 12.4 instead of 10.9 for 8
// sequences of 500 and 4 rows.
constexpr int kCombineRows = 4, kCombineWarps = 8;

template <typename T, int HD>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const __grid_constant__ TreeArgs p) {
  constexpr int R = kCombineRows, ZS = 32 / R, DPL = HD / 32;
  __shared__ __align__(16) float s_o[kCombineWarps][R][HD];
  __shared__ float s_m[kCombineWarps][R], s_l[kCombineWarps][R];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 a = p.desc[2 * c], b = p.desc[2 * c + 1];
  const int r0 = blockIdx.y * R, rows = min(R, a.x - r0);
  if (rows <= 0) return;
  const int n = b.y - b.x + 1;
  auto slot = [&](int z) { return static_cast<size_t>(z == 0 ? b.z : 2 * (b.x + z)) * p.tile_rows + r0; };
  // statistics: a lane has row lane % R of the (lane / R)-th of ZS partials
  const int row = lane & (R - 1), zi = lane / R;
  float m = -INFINITY, l = 0.f, acc[R][DPL] = {};
  auto stats = [&](int k) {  // of this warp's partials from the (ZS k)-th on
    const int z = warp + kCombineWarps * (ZS * k + zi);
    return z < n && row < rows ? *reinterpret_cast<const float2*>(p.part_ml + (slot(z) + row) * 2)
                               : make_float2(-INFINITY, 0.f);
  };
  float2 next = stats(0);
#pragma unroll 1
  for (int k = 0; warp + kCombineWarps * ZS * k < n; ++k) {
    const float2 ml = next;
    next = stats(k + 1);
    float top = fmaxf(ml.x, m);
#pragma unroll
    for (int o = R; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float alpha = merge_weight(m, top), wz = merge_weight(ml.x, top);
    m = top;
    float add = wz * ml.y;
#pragma unroll
    for (int o = R; o < 32; o <<= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
    l = l * alpha + add;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float f = __shfl_sync(0xffffffffu, alpha, r);
#pragma unroll
      for (int d = 0; d < DPL; ++d) acc[r][d] *= f;
    }
#pragma unroll
    for (int i = 0; i < ZS; ++i) {
      const int z = warp + kCombineWarps * (ZS * k + i);
      if (z >= n) break;
      const float* from = p.part_o + slot(z) * HD + lane * DPL;
      float v[R][DPL];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool there = r < rows;
        if constexpr (DPL == 4) {
          const float4 x = there ? load4(from + r * HD) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
        } else {
          const float2 x = there ? *reinterpret_cast<const float2*>(from + r * HD) : make_float2(0.f, 0.f);
          v[r][0] = x.x, v[r][1] = x.y;
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = __shfl_sync(0xffffffffu, wz, i * R + r);
#pragma unroll
        for (int d = 0; d < DPL; ++d) acc[r][d] = fmaf(f, v[r][d], acc[r][d]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int d = 0; d < DPL; ++d) s_o[warp][r][lane * DPL + d] = acc[r][d];
  if (lane < R) {
    s_m[warp][lane] = m;
    s_l[warp][lane] = l;
  }
  __syncthreads();
  static_assert(kCombineWarps >= R, "a warp a row");
  const int r = warp;
  if (r >= rows) return;
  float M = -INFINITY, L = 0.f, out[DPL] = {};
#pragma unroll
  for (int k = 0; k < kCombineWarps; ++k) M = fmaxf(M, s_m[k][r]);
#pragma unroll
  for (int k = 0; k < kCombineWarps; ++k) {
    const float f = merge_weight(s_m[k][r], M);
    L = fmaf(f, s_l[k][r], L);
#pragma unroll
    for (int d = 0; d < DPL; ++d) out[d] = fmaf(f, s_o[k][r][lane * DPL + d], out[d]);
  }
  const float sc = merge_scale(L);
  const int at = a.z + r0 + r;
  T* dst = static_cast<T*>(p.o) + (a.y + at / p.g) * p.o_rs + (a.w * p.g + at % p.g) * p.o_hs + lane * DPL;
#pragma unroll
  for (int d = 0; d < DPL; d += 2) {
    const float x = L == 0.f ? 0.f : out[d] * sc, y = L == 0.f ? 0.f : out[d + 1] * sc;
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint32_t*>(dst + d) = pack_bf16x2(x, y);
    else
      *reinterpret_cast<float2*>(dst + d) = make_float2(x, y);
  }
}

// The same for the tcgen05 kernel's partials, up to 256 rows each, stored [quad of
// columns][row]: an item is 32 rows and eight quads of a cut unit, a warp a quad,
// so that every load is 512 bytes side by side.  Every block counts all units'
// items (one round trip) and takes its share.  The case of one sequence of 40000
// tokens, 19 partials of 183 rows a unit, takes 51.5 us with this merge; with a
// block a possible item (four rounds of blocks, most of them empty), which read
// the maxima first, 58.5.  Batches of 2, 4, 8 partials: 55.5, 51.5, 50.0, and for
// padded batches (2 or 3 a unit) 64.4, 64.3, 67.1.
constexpr int kCombineQuads = 8, kCombineThreads = kCombineQuads * 32;
constexpr int kCombineBlocks = 8;  // per SM
constexpr int kCombineBatch = 4;   // partials read at once
static_assert(kSmBudget <= kCombineThreads, "a thread a run");

template <int HD>
__global__ void __launch_bounds__(kCombineThreads) tree_combine_quads_kernel(const __grid_constant__ TreeArgs p, int runs) {
  constexpr int GROUPS = HD / 4 / kCombineQuads;  // of quads
  __shared__ int s_warp[kCombineThreads / 32], s_end[kCombineThreads];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // thread t: the items of the unit that CTA t + 1's start cuts first, and of those before
  int end = static_cast<int>(threadIdx.x) + 1 < runs ? (p.desc[2 * (threadIdx.x + 1)].x + 31) / 32 * GROUPS : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += u;
  }
  if (lane == 31) s_warp[warp] = end;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int k = 0; k < kCombineThreads / 32; ++k) {
    if (k == warp) end += total;
    total += s_warp[k];
  }
  s_end[threadIdx.x] = end;
  __syncthreads();
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int lo = -1, hi = kCombineThreads - 1;  // the first unit that ends past the item
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_end[mid] > item)
        hi = mid;
      else
        lo = mid;
    }
    const int4 a = p.desc[2 * (hi + 1)], b = p.desc[2 * (hi + 1) + 1];
    const int at = item - (hi > 0 ? s_end[hi - 1] : 0);
    const int row = at / GROUPS * 32 + lane, r = min(row, a.x - 1);
    const int quad = at % GROUPS * kCombineQuads + warp;
    const int n = b.y - b.x + 1;
    auto slot = [&](int z) { return static_cast<size_t>(z == 0 ? b.z : 2 * (b.x + z)) * p.tile_rows; };
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int z0 = 0; z0 < n; z0 += kCombineBatch) {
      float2 ml[kCombineBatch];
      float4 v[kCombineBatch];
#pragma unroll
      for (int z = 0; z < kCombineBatch; ++z) {
        const size_t at_z = slot(min(z0 + z, n - 1));  // (no branch between the loads)
        ml[z] = *reinterpret_cast<const float2*>(p.part_ml + (at_z + r) * 2);
        v[z] = load4(p.part_o + at_z * HD + (quad * p.tile_rows + r) * 4);
        if (z0 + z >= n) ml[z] = make_float2(-INFINITY, 0.f);
      }
      float top = M;
#pragma unroll
      for (int z = 0; z < kCombineBatch; ++z) top = fmaxf(top, ml[z].x);
      const float alpha = merge_weight(M, top);
      M = top;
      L *= alpha;
      acc = make_float4(acc.x * alpha, acc.y * alpha, acc.z * alpha, acc.w * alpha);
#pragma unroll
      for (int z = 0; z < kCombineBatch; ++z) {
        const bool there = z0 + z < n;
        const float wz = there ? merge_weight(ml[z].x, top) : 0.f;
        L = fmaf(wz, ml[z].y, L);
        acc.x = fmaf(wz, there ? v[z].x : 0.f, acc.x);
        acc.y = fmaf(wz, there ? v[z].y : 0.f, acc.y);
        acc.z = fmaf(wz, there ? v[z].z : 0.f, acc.z);
        acc.w = fmaf(wz, there ? v[z].w : 0.f, acc.w);
      }
    }
    if (row >= a.x) continue;
    const float sc = merge_scale(L);
    if (L == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int m = a.z + r;
    store4(static_cast<__nv_bfloat16*>(p.o) + (a.y + m / p.g) * p.o_rs + (a.w * p.g + m % p.g) * p.o_hs + quad * 4,
           make_float4(acc.x * sc, acc.y * sc, acc.z * sc, acc.w * sc));
  }
}

// --------------------------------------------------------------- launches --
// A kernel's geometry: CTAs per SM, rows of a tile, keys of a block.
struct Plan {
  int ctas_per_sm, tile_rows, kb, unit_cost, w_full, w_half;
};

// bf16 rows that fit one or, for head size 64, two row tiles of the warps' matrix
// instructions take the few-rows kernel, more the tcgen05 one.  Both sides
// (few-rows, tcgen05; us; 8 key/value heads, groups of 4):
//   sequences x tokens       32 x 8000      1 x 40000     8 x 500
//   head size 128, 16 rows   167.9  167.3   36.8  39.8    12.1  14.8
//                  20 rows   180.2  168.1   42.3  41.2    15.1  15.0
//                  32 rows   186.5  169.0   44.5  40.7    17.0  15.3
//   head size 64,  16 rows    93.5  100.2   19.1  26.7     9.2  13.4
//                  32 rows   107.3  101.0   25.6  27.1    12.5  13.8
//                  64 rows   199.5  101.8   37.2  27.6    16.8  14.8
// Two row tiles for head size 64 and 16 rows: 105.1, 33.8, 11.7 (chunks of 16).
// A unit's start is worth 2 to 8 blocks without a difference above 2 %, and so are
// weights of 3:2 to 2:1 of a block's full and half tiles.
Plan plan_of(int dtype, int g, int hd, int max_nodes) {
  const int rows = max_nodes * g;
  if (dtype == SPECFOLD_BF16) {
    if (rows > (hd == 128 ? 16 : 32)) return {1, kTreeTcRows, kTreeTcKeys, 5, 5, 3};
    return {Few<128, 1>::CTAS, rows <= 16 ? 16 : 32, kFewKeys, 2, 1, 1};
  }
  return {Simt<128>::CTAS, Simt<128>::RT, kFewKeys, 1, 1, 1};
}

int tree_start(void (*kernel)(TreeArgs), int smem, const TreeArgs& a, int grid, cudaStream_t st) {
  if (const int rc = smem_limit_once(kernel, smem)) return rc;
  launch_k(kernel, dim3(grid), dim3(kThreads), smem, st, a);
  count_launch();
  return check_launch();
}

template <typename T, int HD>
int tree_go(const TreeAttnCall& c, const Plan& pl, cudaStream_t st) {
  TreeArgs a;
  memset(&a, 0, sizeof(a));
  a.q = c.q.ptr;
  a.q_rs = c.q.row_stride;
  a.q_hs = c.q.head_stride;
  a.o = c.o.ptr;
  a.o_rs = c.o.row_stride;
  a.o_hs = c.o.head_stride;
  a.cache = c.cache;
  a.parent = c.parent;
  a.batch = c.batch;
  a.max_nodes = c.max_nodes;
  a.most_tokens = 0xffffffffu;
  a.n_kv = c.n_kv;
  a.g = c.n_q / c.n_kv;
  a.tile_rows = pl.tile_rows;
  a.kb = pl.kb;
  a.unit_cost = pl.unit_cost;
  a.w_full = pl.w_full;
  a.w_half = pl.w_half;
  a.sl2 = static_cast<float>(1.4426950408889634 * (c.scale > 0.f ? c.scale : 1.0 / std::sqrt(static_cast<double>(HD))));
  uint8_t* ws = static_cast<uint8_t*>(c.ws);
  a.status = reinterpret_cast<uint32_t*>(ws);
  const int slots = 2 * kSmBudget * pl.ctas_per_sm;
  a.desc = reinterpret_cast<int4*>(ws + 256);
  a.part_ml = reinterpret_cast<float*>(a.desc + slots);
  a.part_o = a.part_ml + static_cast<size_t>(slots) * pl.tile_rows * 2;
  const int grid = std::min(num_sms(), kSmBudget) * pl.ctas_per_sm;
  int rc;
  if constexpr (sizeof(T) == 2) {
    if (pl.tile_rows == 16)
      rc = tree_start(tree_attn_few_kernel<HD, 1>, Few<HD, 1>::SMEM, a, grid, st);
    else if (HD == 64 && pl.tile_rows == 32)
      rc = tree_start(tree_attn_few_kernel<64, 2>, Few<64, 2>::SMEM, a, grid, st);
    else
      rc = launch_tree_tc(a, HD, grid, st);
  } else {
    rc = tree_start(tree_attn_simt_kernel<HD>, Simt<HD>::SMEM, a, grid, st);
  }
  if (rc) return rc;
  if (grid == 1) return SPECFOLD_OK;
  if (sizeof(T) == 2 && pl.tile_rows == kTreeTcRows)
    launch_k(tree_combine_quads_kernel<HD>, dim3(kCombineBlocks * num_sms()), dim3(kCombineThreads), 0, st, a, grid);
  else
    launch_k(tree_combine_kernel<T, HD>, dim3(grid - 1, (std::min(pl.tile_rows, a.max_nodes * a.g) + kCombineRows - 1) / kCombineRows),
             dim3(kCombineWarps * 32), 0, st, a);
  count_launch();
  return check_launch();
}

}  // namespace

size_t tree_attn_ws_bytes(int dtype, int n_q, int n_kv, int hd, int max_nodes) {
  const Plan pl = plan_of(dtype, n_q / n_kv, hd, max_nodes);
  const size_t slots = 2 * static_cast<size_t>(kSmBudget) * pl.ctas_per_sm;
  return 256 + slots * (sizeof(int4) + static_cast<size_t>(pl.tile_rows) * (hd + 2) * sizeof(float));
}

int launch_tree_attention(const TreeAttnCall& c, cudaStream_t st) {
  const Plan pl = plan_of(c.dtype, c.n_q / c.n_kv, c.hd, c.max_nodes);
  if (c.dtype == SPECFOLD_BF16)
    return c.hd == 128 ? tree_go<__nv_bfloat16, 128>(c, pl, st) : tree_go<__nv_bfloat16, 64>(c, pl, st);
  return c.hd == 128 ? tree_go<float, 128>(c, pl, st) : tree_go<float, 64>(c, pl, st);
}

}  // namespace sf

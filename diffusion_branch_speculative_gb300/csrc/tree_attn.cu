// Attention of drafted rows over a paged cache and their tree
// (specfold_tree_attention): the kernel on the CUDA cores and the merge of
// split units.  tree_sched.cuh has the decomposition.
#include "tree_sched.cuh"

#include <algorithm>
#include <cmath>
#include <cstring>

namespace sf {
namespace {

constexpr int kThreads = 128;  // 4 warps, each with its own chunks of keys
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 16;     // keys of a warp's step
constexpr int kSmBudget = 160; // SMs the workspace is sized for (>= one GB300)

SF_DEV float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
SF_DEV float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}
SF_DEV void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
SF_DEV void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Weight of a partial with maximum m in a merge with maximum M: 1 where they
// are equal, -inf included (a partial that saw nothing holds zeros, and one
// whose scores are NaN keeps its NaN).
SF_DEV float merge_weight(float m, float M) { return m == M ? 1.f : ex2(m - M); }
// The output of a row with sum l: zeros where nothing was seen.
SF_DEV float merge_scale(float l) { return l == 0.f ? 0.f : 1.f / l; }

// ------------------------------------------------------------ CUDA cores --
// Tiles of RT rows (row m = node m / g, head m % g of the group).  Every warp
// streams its own chunks of 16 keys through a private ring of asynchronous
// copies, with its own running maximum and sum, so the loop has no block-wide
// barrier; the four warps merge once per piece.
//   scores: lane = (key, half of the dimensions), the row's query broadcast
//           from shared memory, the halves joined by one shuffle;
//   output: lane = dimensions, the probabilities broadcast.
// A chunk's 16-byte pieces are stored with their index xored with the row's low
// three bits, so that eight rows read at one place never share a bank.
template <typename T, int HD>
struct Simt {
  static constexpr int RT = 8;
  static constexpr int STAGES = 2;
  static constexpr int ROW = HD * sizeof(T);        // bytes of a key
  static constexpr int CPR = ROW / 16;              // 16-byte pieces of a key
  static constexpr int STAGE = 2 * kChunk * ROW;    // keys, then values
  static constexpr int RING = STAGES * STAGE;       // of one warp
  static constexpr int MERGE = RT * (HD + 2) * 4;   // of one warp, over its ring
  static constexpr int OFF_Q = kWarps * (RING > MERGE ? RING : MERGE);
  static constexpr int OFF_P = OFF_Q + RT * HD * 4;
  static constexpr int SMEM = OFF_P + kWarps * kChunk * RT * 4;
};

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) tree_attn_simt_kernel(const __grid_constant__ TreeArgs p) {
  using C = Simt<T, HD>;
  constexpr int RT = C::RT, DPL = HD / 32;  // dimensions of the output a lane holds
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ TreeLocate loc;
  __shared__ int16_t s_parent[SPECFOLD_MAX_TREE];
  __shared__ uint32_t s_sees[RT][SPECFOLD_MAX_TREE / 32];  // a tile row's ancestors and itself
  __shared__ int s_dead[RT];                               // padding rows
  pdl_wait();
  pdl_trigger();
  TreeWalk w;
  if (!tree_locate<kThreads>(p, loc, w)) {
    if (threadIdx.x == 0) tree_describe_none(p);
    return;
  }
  if (threadIdx.x == 0) tree_describe(p, w, loc.per, loc.lo);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * (C::RING > C::MERGE ? C::RING : C::MERGE);
  float* s_q = reinterpret_cast<float*>(smem + C::OFF_Q);
  float* s_p = reinterpret_cast<float*>(smem + C::OFF_P) + warp * kChunk * RT;
  const T* qp = static_cast<const T*>(p.q);
  T* op = static_cast<T*>(p.o);

  for (bool first = true; w.left > 0; first = false, w.next(p)) {
    const int h = w.head(), m0 = tree_m0(p, w), rows = tree_tile_rows(p, w);
    const int len = w.q.ctx + w.q.n, key_lo = w.b0 * p.kb;
    const int key_hi = min(static_cast<long long>(len), static_cast<long long>(w.b0 + w.blocks()) * p.kb);
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

    // this warp's chunks: key_lo + 16 * (warp + 4 i)
    const int chunks = (key_hi - key_lo + kChunk - 1) / kChunk;
    const int mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
    auto key_of = [&](int i) { return key_lo + kChunk * (warp + kWarps * i); };
    auto slot_of = [&](int i) {  // lanes 0..15: pool tokens of chunk i's keys
      const int tok = key_of(i) + (lane & (kChunk - 1));
      return i < mine && tok < key_hi ? tree_pool_token(p, w.s, tok) : -1;
    };
    auto load = [&](int i, int slot) {
      if (i < mine) {
        uint8_t* st = ring + (i % C::STAGES) * C::STAGE;
#pragma unroll
        for (int it = 0; it < 2 * kChunk * C::CPR / 32; ++it) {
          const int idx = it * 32 + lane;
          const int c = idx % C::CPR, key = (idx / C::CPR) % kChunk, is_v = idx / (C::CPR * kChunk);
          const int tk = __shfl_sync(0xffffffffu, slot, key);
          const T* src = is_v ? static_cast<const T*>(p.cache.v) + tk * p.cache.v_token_stride + h * p.cache.v_head_stride
                              : static_cast<const T*>(p.cache.k) + tk * p.cache.k_token_stride + h * p.cache.k_head_stride;
          if (tk < 0) src = static_cast<const T*>(p.cache.k);  // any valid address: nothing is read
          cp_async16(smem_u32(st + is_v * kChunk * C::ROW + key * C::ROW + ((c ^ (key & 7)) << 4)),
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
    for (int i = 0; i < mine; ++i) {
      load(i + C::STAGES - 1, slot);
      slot = slot_of(i + C::STAGES);
      cp_async_wait<C::STAGES - 1>();
      __syncwarp();
      const uint8_t* sk = ring + (i % C::STAGES) * C::STAGE;
      const uint8_t* sv = sk + kChunk * C::ROW;
      const int key = lane & (kChunk - 1), half = lane / kChunk;
      float s[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) s[r] = 0.f;
#pragma unroll 4
      for (int d = 0; d < HD / 2; d += 4) {
        const float4 k4 = load4(at(sk, key, half * (HD / 2) + d));
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float4 q4 = load4(s_q + r * HD + half * (HD / 2) + d);
          s[r] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[r]))));
        }
      }
      const int tok = key_of(i) + key, e = tok - w.q.ctx;
      const bool tail = key_of(i) + kChunk > w.q.ctx;  // holds tokens that not every row sees
      float pr[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        s[r] += __shfl_xor_sync(0xffffffffu, s[r], kChunk);
        bool see = !s_dead[r];
        if (tail) see = see && tok < key_hi && (e < 0 || (s_sees[r][(e >> 5) & 7] >> (e & 31) & 1u));
        s[r] = see ? s[r] * p.sl2 : -INFINITY;
        float m = s[r];
#pragma unroll
        for (int o = kChunk / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
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
      if (half == 0) {
        store4(s_p + key * RT, make_float4(pr[0], pr[1], pr[2], pr[3]));
        store4(s_p + key * RT + 4, make_float4(pr[4], pr[5], pr[6], pr[7]));
      }
      __syncwarp();
#pragma unroll 4
      for (int k = 0; k < kChunk; ++k) {
        float v[DPL];
        const T* vp = at(sv, k, lane * DPL);
#pragma unroll
        for (int d = 0; d < DPL; ++d) v[d] = static_cast<float>(vp[d]);
        const float4 pa = load4(s_p + k * RT), pb = load4(s_p + k * RT + 4);
        const float pk[RT] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          // a token the row does not see adds nothing, whatever its value
          if (!tail || pk[r] != 0.f) {
#pragma unroll
            for (int d = 0; d < DPL; ++d) acc[r][d] = fmaf(pk[r], v[d], acc[r][d]);
          }
        }
      }
      __syncwarp();  // the stage and the probabilities may be overwritten
    }
    cp_async_wait<0>();
    __syncwarp();

    // the warps' merge: each writes (o, m, l) over its own ring
    float* mo = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float ls = l[r];
#pragma unroll
      for (int o = kChunk / 2; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
#pragma unroll
      for (int d = 0; d < DPL; ++d) mo[r * HD + lane * DPL + d] = acc[r][d];
      if (lane == 0) {
        mo[RT * HD + 2 * r] = mx[r];
        mo[RT * HD + 2 * r + 1] = ls;
      }
    }
    __syncthreads();
    const bool whole = w.whole();
    const size_t ps = static_cast<size_t>(tree_slot(first)) * p.tile_rows;
    constexpr int WSTEP = (C::RING > C::MERGE ? C::RING : C::MERGE) / 4;
    const float* mw = reinterpret_cast<const float*>(smem);
    for (int i = threadIdx.x; i < rows * (HD / 4); i += kThreads) {
      const int r = i / (HD / 4), d = (i % (HD / 4)) * 4;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) M = fmaxf(M, mw[k * WSTEP + RT * HD + 2 * r]);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float wk = merge_weight(mw[k * WSTEP + RT * HD + 2 * r], M);
        const float4 v = load4(mw + k * WSTEP + r * HD + d);
        L = fmaf(wk, mw[k * WSTEP + RT * HD + 2 * r + 1], L);
        a.x = fmaf(wk, v.x, a.x);
        a.y = fmaf(wk, v.y, a.y);
        a.z = fmaf(wk, v.z, a.z);
        a.w = fmaf(wk, v.w, a.w);
      }
      if (whole) {
        const int m = m0 + r;
        const float sc = merge_scale(L);
        if (L == 0.f) a = make_float4(0.f, 0.f, 0.f, 0.f);
        store4(op + (w.q.row0 + m / p.g) * p.o_rs + (h * p.g + m % p.g) * p.o_hs + d,
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
}

// ---------------------------------------------------------------- combine --
// Merges the partials of cut units: block (c, y) has the unit that CTA c's
// start cuts first, one warp per row.  The partials of one unit lie at its
// first CTA's slot and at the first slots of the CTAs after it.
constexpr int kCombineRows = 8;

template <typename T, int HD>
__global__ void __launch_bounds__(kCombineRows * 32) tree_combine_kernel(const __grid_constant__ TreeArgs p) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x + 1;
  const int4 a = p.desc[2 * c], b = p.desc[2 * c + 1];
  const int r = blockIdx.y * kCombineRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= a.x) return;
  constexpr int DPL = HD / 32;
  const int n = b.y - b.x + 1;
  auto slot = [&](int z) { return static_cast<size_t>(z == 0 ? b.z : 2 * (b.x + z)) * p.tile_rows + r; };
  float M = -INFINITY;
  for (int z = lane; z < n; z += 32) M = fmaxf(M, p.part_ml[slot(z) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f, acc[DPL] = {};
  for (int z0 = 0; z0 < n; z0 += 32) {
    float wz = 0.f, lz = 0.f;
    if (z0 + lane < n) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + slot(z0 + lane) * 2);
      wz = merge_weight(ml.x, M);
      lz = ml.y * wz;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lz += __shfl_xor_sync(0xffffffffu, lz, o);
    L += lz;
    const int m = min(32, n - z0);
#pragma unroll 4
    for (int z = 0; z < m; ++z) {
      const float wv = __shfl_sync(0xffffffffu, wz, z);
      const float* v = p.part_o + slot(z0 + z) * HD + lane * DPL;
      if constexpr (DPL == 4) {
        const float4 x = load4(v);
        acc[0] = fmaf(wv, x.x, acc[0]);
        acc[1] = fmaf(wv, x.y, acc[1]);
        acc[2] = fmaf(wv, x.z, acc[2]);
        acc[3] = fmaf(wv, x.w, acc[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(v);
        acc[0] = fmaf(wv, x.x, acc[0]);
        acc[1] = fmaf(wv, x.y, acc[1]);
      }
    }
  }
  const float sc = merge_scale(L);
  const int m = a.z + r;
  T* dst = static_cast<T*>(p.o) + (a.y + m / p.g) * p.o_rs + (a.w * p.g + m % p.g) * p.o_hs + lane * DPL;
#pragma unroll
  for (int d = 0; d < DPL; d += 2) {
    const float x = L == 0.f ? 0.f : acc[d] * sc, y = L == 0.f ? 0.f : acc[d + 1] * sc;
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint32_t*>(dst + d) = pack_bf16x2(x, y);
    else
      *reinterpret_cast<float2*>(dst + d) = make_float2(x, y);
  }
}

// --------------------------------------------------------------- launches --
// A kernel's geometry: CTAs per SM, rows of a tile, keys of a block.
struct Plan {
  int ctas_per_sm, tile_mul, tile_per, tile_rows, kb;
};

Plan plan_of(int dtype, int g, int hd, int max_nodes) {
  (void)dtype;
  (void)hd;
  (void)max_nodes;
  return {1, g, 8, 8, 4 * kChunk};
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
  a.n_kv = c.n_kv;
  a.g = c.n_q / c.n_kv;
  a.tile_mul = pl.tile_mul;
  a.tile_per = pl.tile_per;
  a.tile_rows = pl.tile_rows;
  a.kb = pl.kb;
  a.sl2 = static_cast<float>(1.4426950408889634 * (c.scale > 0.f ? c.scale : 1.0 / std::sqrt(static_cast<double>(HD))));
  uint8_t* ws = static_cast<uint8_t*>(c.ws);
  a.status = reinterpret_cast<uint32_t*>(ws);
  const int slots = 2 * kSmBudget * pl.ctas_per_sm;
  a.desc = reinterpret_cast<int4*>(ws + 256);
  a.part_ml = reinterpret_cast<float*>(a.desc + slots);
  a.part_o = a.part_ml + static_cast<size_t>(slots) * pl.tile_rows * 2;
  const int grid = std::min(num_sms(), kSmBudget) * pl.ctas_per_sm;
  using C = Simt<T, HD>;
  if (const int rc = smem_limit_once(tree_attn_simt_kernel<T, HD>, C::SMEM)) return rc;
  launch_k(tree_attn_simt_kernel<T, HD>, dim3(grid), dim3(kThreads), C::SMEM, st, a);
  count_launch();
  if (const int rc = check_launch()) return rc;
  if (grid == 1) return SPECFOLD_OK;
  launch_k(tree_combine_kernel<T, HD>, dim3(grid - 1, (pl.tile_rows + kCombineRows - 1) / kCombineRows),
           dim3(kCombineRows * 32), 0, st, a);
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

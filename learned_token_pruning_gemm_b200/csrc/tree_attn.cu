// tg_tree_attention: a tree of drafted tokens attends over the compacted cache
// (MarkTechPost page on TokenGate, section "Comment déployer TokenGate ?": generation
// runs on the cache that the pruned prefill leaves; section "Qu'est-ce que l'attention
// gérée par des tokens ?": key-score bias and per-head temperature). Drafted token t
// of sequence b sees every cache row j < cache_len[b] and the drafted tokens whose bit
// is set in tree_mask[b][t]:
//     z_j = q . k_j / (sqrt(dh) tau_h) + g_h s_j,   O = sum_j softmax_j(z) v_j.
//
// The cache is read once per KV head and pair of row tiles (up to 256 rows; whole tokens, so
// 192 for 64 tokens of three heads) and serves the drafted tokens and query heads in it: with
// R = (tokens) x (group) rows this is a [R x dh] x [dh x len] product and back. Here the rows
// are packed into M = 128 tiles (row r is token r / G, head r % G) and both products run on the
// tensor cores with accumulators in TMEM; up to 16 rows over codes take the kernel of
// tree_rows.cu instead. Work is split as tree.cuh says, in units of 128 cache rows; what a CTA
// has of an item it leaves as partials (max, sum, O), and the kernel at the end adds the
// partials up in CTA order, so results do not depend on timing, and brings in the drafted rows
// that each token sees.
//
// A CTA has two sides, each with its own softmax warps, S buffers and O in TMEM. The sides take
// the two row tiles of an item, which then share every K and V tile and its widening; of an item
// of one row tile they take half of every unit's keys each, and each leaves a partial. A job is
// 64 keys of a side; it has two S buffers, so that its products run while the softmax is at the
// job before.
//
// Per CTA, pipelines run over the units:
//   warp 0       K tiles by TMA (bf16: into the operand ring; codes: K and V codes into a
//                raw ring). A bf16 tile that ends inside is copied row by row.
//   warp 3       V tiles likewise (bf16 cache)
//   warp 2       the rows' queries, and per key: score, scales (a ring of four tiles)
//   warps 20-23  codes only: widen the raw tiles into fp16 operand tiles. Codes are exact in
//                fp16, so scales are applied in fp32, to logits and weights.
//   warp 1       MMA issuer (one thread), the sides in turn: S_0, S_1, then PV_k, S_{k + 2}, ..;
//                S = Q K^T into one of the side's TMEM buffers, O += P V with P read from TMEM
//                (it overwrites S) and V as an MN-major shared-memory operand.
//   warps 4-19   softmax, 16 rows a warp, those with rows only: logits in the log2 domain
//                less the row's running reference, which moves only when one exceeds it by more
//                than it may (O is then rescaled in TMEM).
//
// What bounds it: the softmax's instructions (57% of the issue slots are busy, at 24 warps an SM;
// the tensor pipe 30% of the time) and, with few rows, the way of a unit through the roles. 2 x 64
// tokens of 32 heads over 65500 int8 rows of four heads: 227 us (0.61 PFLOP/s, 84.5 us at a plain
// GEMM's rate; 200 us without the combining kernel); 8 x 13 tokens of 16 heads over 50 thousand
// bf16 rows of eight: 57 us (31.3 us at a plain copy's rate). Steps that made it so, on the long
// case: one row tile a CTA 379 us; two tiles that share K, V and their widening 318; queries, keys
// and values waiting less for one another 246; one thread chosen by elect.sync for the products (a
// lane picked by its number costs 80 to 110 cycles an MMA, an elected one 25 to 45) and jobs of 64
// keys 253; 16 rows a warp 229; streams of eight lanes in the combining kernel 224; the reference
// taken off rounded logits, and scores held to a finite product, 227.
//
// The codes variants hold 80 registers at 768 threads and spill 100 to 124 bytes (stores; loads 172
// to 188), most likely around the 32 logits of a job; the bf16 ones (96 registers) 4 to 12.
// Other shapes, floors at a plain copy's and GEMM's rate in brackets: 13 tokens of 16 heads over
// 8 x 10721 rows of eight: bf16 71 us (54), int8 102 us (28), int8 of head dim 64 92 us (14): one
// row tile of 26 rows, whose softmax warps share one scheduler, and for codes one V tile, so
// that the next V is not widened before the last product with this one; 64 tokens of 16 heads of 64
// over 4 x 10000 int8 rows 61 us (7), 32 tokens over 8 x 1000 bf16 rows 28 us (5.5): about half in the
// combining kernel, which takes every drafted row again for every token and head.
//
// Weights are rounded for the second product, to bf16 beside bf16 values (a product's operands
// have one type, and fp16 lacks the values' range) and to fp16 beside codes. Of the output, in
// the 2-norm: 0.0021 and 0.0016 from the 64-bit form, where storing it in bf16 alone is 0.0016.
//
// A side's S_k is issued after its PV_{k - 2}, and products end in the order they are issued:
// when S_k is there, all but PV_{k - 1} are done, so no parity wait is passed by.
#include "tree.cuh"

namespace {

using tg::TreeArgs;
using tg::bf16_hi;
using tg::bf16_lo;
using tg::kLog2e;
using tg::wait;

constexpr int kBM = 128;           // rows of a row tile
constexpr int kBN = 128;           // keys of a unit
constexpr int kJob = 64;           // keys of a job
constexpr int kMaxDraft = 64;
constexpr int kKeyStages = 4;
constexpr int kSideWarps = 8;      // softmax warps of a side
constexpr int kConvWarps = 4;
constexpr int kMaxCtas = 148;      // one per SM
constexpr uint32_t kHalfBytes = kBN * 128;  // 64 columns of 128 rows, bf16, 128-byte swizzle
constexpr uint32_t kTmemCols = 512, kColO = 256;   // S at 0 and 128, O at 256 and 384

template <int DH, bool kQ>
struct Cfg {
  static constexpr int kHalves = DH / 64;
  static constexpr int kK = DH == 128 ? 2 : 4;                           // K operand tiles
  static constexpr int kV = DH == 128 ? (kQ ? 1 : 2) : 4;                // V operand tiles
  static constexpr int kRaw = kQ ? (DH == 128 ? 3 : 4) : 1;              // raw tiles of codes
  static constexpr int kRawBytes = kQ ? kBN * DH : 16;
  static constexpr int kThreads = 128 + 2 * kSideWarps * 32 + (kQ ? kConvWarps * 32 : 0);
  static constexpr int kFullArrivals = kQ ? kConvWarps : 1;              // a K or V tile is ready
};

template <int DH, bool kQ>
struct TreeSmem {
  using C = Cfg<DH, kQ>;
  uint8_t q[2][C::kHalves][kHalfBytes];   // by side
  uint8_t k[C::kK][C::kHalves][kHalfBytes];
  uint8_t v[C::kV][C::kHalves][kHalfBytes];
  uint8_t raw[C::kRaw][C::kRawBytes];
  // score; codes: scores and key scales of two keys side by side (2 x kBN), then log2 of the value
  // scale, then its inverse
  alignas(16) float key[kKeyStages][kQ ? 4 : 1][kBN];
  int base[tg::kTreeMaxBatch + 1];
  int len[tg::kTreeMaxBatch];
  uint8_t dl[tg::kTreeMaxBatch];
  uint64_t q_full, q_ready, q_empty;   // landed; in fp16 (codes); every S of the item done
  uint64_t k_full[C::kK], k_empty[C::kK];
  uint64_t v_full[C::kV], v_empty[C::kV];
  uint64_t raw_full[C::kRaw], raw_empty[C::kRaw];
  uint64_t b_full[kKeyStages], b_empty[kKeyStages];
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2], o_free[2];   // by side, and by buffer
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ bool all_alive(bool a) { return __all_sync(0xFFFFFFFFu, a); }

// The order in which the tiles of a quantised cache pass, K two units ahead of V as S is of O:
// K_0, K_1, V_0, K_2, V_1, .., K_{n-1}, V_{n-2}, V_{n-1}. Whether turn i is a V.
__device__ __forceinline__ bool value_turn(int i, int n) { return i == 2 * n - 1 || (i > 0 && (i & 1) == 0); }

// Walks a CTA's units in order: the unit's sequence, KV head, pair of row tiles and place
// among its item's units. two: the pair's second tile is there.
struct Cursor {
  int u, u1, b, item, n_items, kvh, pair, j, nt, len, tiles;
  bool two;
  __device__ __forceinline__ void load_seq(const TreeArgs& A, const tg::TreeSeqs& s) {
    len = s.len[b];
    tiles = tg::row_tiles(A, s.dl[b]);
    nt = (len + kBN - 1) / kBN;
    n_items = A.n_hkv * ((tiles + 1) / 2);
  }
  __device__ __forceinline__ void split_item(const TreeArgs& A) {
    const int pairs = (tiles + 1) / 2;
    kvh = item / pairs;
    pair = item - kvh * pairs;
    two = 2 * pair + 1 < tiles;
  }
  __device__ __forceinline__ void start(const TreeArgs& A, const tg::TreeSeqs& s, int first, int n) {
    u = first;
    u1 = first + n;
    b = tg::sequence_of(A, s, u);
    load_seq(A, s);
    item = (u - s.base[b]) / nt;
    j = u - s.base[b] - item * nt;
    split_item(A);
  }
  __device__ __forceinline__ void advance(const TreeArgs& A, const tg::TreeSeqs& s, int by = 1) {   // by: run() at most
    u += by;
    if ((j += by) < nt || u >= u1) return;
    j = 0;
    if (++item == n_items) {
      item = 0;
      do ++b;
      while (s.base[b + 1] == s.base[b]);   // sequences without units
      load_seq(A, s);
    }
    split_item(A);
  }
  __device__ __forceinline__ int keys() const { return min(kBN, len - j * kBN); }
  // units of the current item from here on within the CTA's share
  __device__ __forceinline__ int run() const { return min(nt - j, u1 - u); }
};

// 16 bytes global -> shared, or 16 zero bytes when !ok (src is not read then)
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// byte offset of 16-byte column c (0 .. dh/8 - 1) of row r in a swizzled operand tile
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (c >> 3) * kHalfBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void fmul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void ffma2(float& d0, float& d1, float a0, float a1, float b0, float b1,
                                      float c0, float c1) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void fadd2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 16 rows by 16 columns, as the 16x256b loads of 64 columns
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_16x256b_x2(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 16 rows by 32 columns: thread l holds (row l/4, column 4i + l%4) in register 2i and
// the same column of row l/4 + 8 in register 2i + 1.
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32"
      " [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// acc += the low (lo) or high (hi) bf16 half of a packed pair, widened exactly
__device__ __forceinline__ void add_bf16_lo(float& acc, uint32_t u) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.bf16 %0, l, %0;\n\t}" : "+f"(acc) : "r"(u));
}
__device__ __forceinline__ void add_bf16_hi(float& acc, uint32_t u) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.bf16 %0, h, %0;\n\t}" : "+f"(acc) : "r"(u));
}
__device__ __forceinline__ void cp4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tg::smem_u32(dst)), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// One lane of a converged warp; the compiler then knows that a single thread goes on.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes;
}
// Instruction descriptor of an fp16 (kF16) or bf16 product: the format fields are 0 for fp16.
template <bool kF16>
constexpr uint32_t idesc(int M, int N, bool b_mn) {
  return tg::idesc_bf16_f32(M, N, false, b_mn) & (kF16 ? ~((1u << 7) | (1u << 10)) : ~0u);
}

template <int DH, int kType>
__global__ void __launch_bounds__(Cfg<DH, kType != TG_BF16>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeArgs A) {
  constexpr bool kQ = kType != TG_BF16;
  using C = Cfg<DH, kQ>;
  using Smem = TreeSmem<DH, kQ>;
  constexpr uint32_t kTileBytes = C::kHalves * kHalfBytes;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (tg::smem_u32(smem_raw) & 1023u)) & 1023u;
  Smem& S = *reinterpret_cast<Smem*>(smem_raw + pad);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = A.group * A.tm;                    // rows in use of a row tile
  const int n_act = (rows + 15) / 16;                 // softmax warps of a side with rows

  if (tid == 0) {
    tg::mbar_init(&S.q_full, 1);
    tg::mbar_init(&S.q_ready, 2 * n_act);
    tg::mbar_init(&S.q_empty, 1);
    for (int s = 0; s < C::kK; ++s) {
      tg::mbar_init(&S.k_full[s], C::kFullArrivals);
      tg::mbar_init(&S.k_empty[s], 1);
    }
    for (int s = 0; s < C::kV; ++s) {
      tg::mbar_init(&S.v_full[s], C::kFullArrivals);
      tg::mbar_init(&S.v_empty[s], 1);
    }
    for (int s = 0; s < C::kRaw; ++s) {
      tg::mbar_init(&S.raw_full[s], 1);
      tg::mbar_init(&S.raw_empty[s], kConvWarps);
    }
    for (int s = 0; s < kKeyStages; ++s) {
      tg::mbar_init(&S.b_full[s], 32);
      tg::mbar_init(&S.b_empty[s], 2 * n_act);
    }
    for (int s = 0; s < 2; ++s) {
      for (int i = 0; i < 2; ++i) {
        tg::mbar_init(&S.s_full[s][i], 1);
        tg::mbar_init(&S.p_full[s][i], n_act);
        tg::mbar_init(&S.o_done[s][i], 1);
      }
      tg::mbar_init(&S.o_free[s], n_act);
    }
    S.abort_flag = 0;
    tg::fence_barrier_init();
    tg::tma_prefetch_desc(&tm_q);
    tg::tma_prefetch_desc(&tm_k);
    tg::tma_prefetch_desc(&tm_v);
  }
  if (warp == 2) {
    tg::tmem_alloc(&S.tmem_base, kTmemCols);
    tg::tmem_relinquish();
  }
  tg::pdl_launch_dependents();
  tg::pdl_wait();   // global memory only from here on
  tg::tc_fence_before();
  const tg::TreeSeqs Q{S.base, S.len, S.dl};
  const tg::Shares share(A, tg::count_units<C::kThreads>(A, Q));
  tg::tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  const int n = share.size(blockIdx.x);
  if (n == 0) {   // uniform: nothing to do here
    if (warp == 2) tg::tmem_dealloc(tmem, kTmemCols);
    return;
  }
  Cursor c;
  c.start(A, Q, share.first(blockIdx.x), n);

  if (!kQ && (warp == 0 || warp == 3)) {
    // ---------------- K (warp 0) or V (warp 3) tiles of a bf16 cache ----------------
    const bool val = warp == 3;
    constexpr int kC = DH / 8;
    const int n_st = val ? C::kV : C::kK;
    uint64_t* full = val ? S.v_full : S.k_full;
    uint64_t* empty = val ? S.v_empty : S.k_empty;
    const CUtensorMap* map = val ? &tm_v : &tm_k;
    const __nv_bfloat16* cache = reinterpret_cast<const __nv_bfloat16*>(val ? A.vc : A.kc);
    int g = 0;
#pragma unroll 1
    for (; g < n; ++g, c.advance(A, Q)) {
      const int s = g % n_st;
      if (g >= n_st &&
          !all_alive(wait(&empty[s], ((g / n_st) - 1) & 1, A.status, &S.abort_flag)))
        break;
      uint8_t* dst = val ? S.v[s % C::kV][0] : S.k[s % C::kK][0];
      const int nv = c.keys();
      if (nv < kBN) {   // V: rows behind the end are zero up to a multiple of 16, as P's columns are
        const int r1 = val ? (nv + 15) & ~15 : nv;
#pragma unroll 1
        for (int i = lane; i < r1 * kC; i += 32) {
          const int r = i / kC, cc = i % kC;
          const int64_t hr = (static_cast<int64_t>(c.b) * A.cap + c.j * kBN + min(r, nv - 1)) * A.n_hkv + c.kvh;
          const bool ok = r < nv && tg::in_bounds(hr, static_cast<int64_t>(A.batch) * A.cap * A.n_hkv, A.status);
          cp16(tg::smem_u32(dst) + tile_off(r, cc), cache + hr * DH + 8 * cc, ok);
        }
        cp_wait_all();
        tg::fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) tg::mbar_arrive(&full[s]);
      } else if (lane == 0) {
        tg::mbar_arrive_expect_tx(&full[s], kTileBytes);
        const int row = static_cast<int>(static_cast<int64_t>(c.b) * A.cap + c.j * kBN);
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
          tg::tma_load_3d(dst + h * kHalfBytes, map, &full[s], 64 * h, row, c.kvh);
      }
      __syncwarp();
    }
    if (S.abort_flag && lane == 0)   // let copies in flight land before the CTA exits
      for (int i = g > n_st ? g - n_st : 0; i < g; ++i)
        wait(&full[i % n_st], (i / n_st) & 1, A.status, nullptr);
    __syncwarp();
  } else if (kQ && warp == 0) {
    // ---------------- codes by TMA ----------------
    if (lane == 0) {
      int r = 0, row = 0, kvh = 0, last_row = 0, last_kvh = 0;   // of the K tile and the one before
#pragma unroll 1
      for (; r < 2 * n; ++r) {
        const bool val = value_turn(r, n);
        if (!val) {
          last_row = row, last_kvh = kvh;
          row = static_cast<int>(static_cast<int64_t>(c.b) * A.cap + c.j * kBN), kvh = c.kvh;
          c.advance(A, Q);
        }
        const bool before = val && r < 2 * n - 1;
        const int s = r % C::kRaw;
        if (r >= C::kRaw && !wait(&S.raw_empty[s], ((r / C::kRaw) - 1) & 1, A.status, &S.abort_flag)) break;
        tg::mbar_arrive_expect_tx(&S.raw_full[s], C::kRawBytes);
        tg::tma_load_3d(S.raw[s], val ? &tm_v : &tm_k, &S.raw_full[s], 0, before ? last_row : row,
                        before ? last_kvh : kvh);
      }
      if (S.abort_flag)
        for (int i = r > C::kRaw ? r - C::kRaw : 0; i < r; ++i)
          wait(&S.raw_full[i % C::kRaw], (i / C::kRaw) & 1, A.status, nullptr);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- queries, and what each key brings besides K and V ----------------
    // The keys' data by small asynchronous copies into their ring, kLag tiles before they are
    // handed on: with two, the copies that go ahead wait for the tile before the last, not for
    // the one at work. Keys behind the end read the last one's place: they are masked.
    constexpr int kLag = kKeyStages - 2;
    Cursor la = c;
    int n_q = 0;
    auto queries = [&](const Cursor& t) {
      if (lane == 0) {
        tg::mbar_arrive_expect_tx(&S.q_full, 2 * C::kHalves * rows * 128);
#pragma unroll
        for (int i = 0; i < 2 * C::kHalves; ++i) {   // one row tile: for either side
          const int side = i / C::kHalves, h = i % C::kHalves, mt = 2 * t.pair + (t.two ? side : 0);
          tg::tma_load_3d(S.q[side][h], &tm_q, &S.q_full, 64 * h, t.kvh * A.group, t.b * A.n_draft + mt * A.tm);
        }
      }
      ++n_q;
      __syncwarp();
    };
    queries(c);
#pragma unroll 1
    for (int g = 0; g < n + kLag; ++g) {
      if (g < n) {
        const int s = g % kKeyStages;
        if (g >= kKeyStages &&
            !all_alive(wait(&S.b_empty[s], ((g / kKeyStages) - 1) & 1, A.status, &S.abort_flag)))
          break;
        const int64_t row0 = static_cast<int64_t>(la.b) * A.cap + la.j * kBN;
        const int last = la.keys() - 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = lane + 32 * i;
          const int64_t row = row0 + min(j, last);
          if (!tg::in_bounds(row, static_cast<int64_t>(A.batch) * A.cap, A.status)) continue;
          float* at = S.key[s][0] + (kQ ? 4 * (j >> 1) + (j & 1) : j);
          cp4(at, A.sc + row);
          if constexpr (kQ) {
            cp4(at + 2, A.ks + row * A.n_hkv + la.kvh);
            cp4(&S.key[s][2][j], A.vs + row * A.n_hkv + la.kvh);
          }
        }
        la.advance(A, Q);
      }
      cp_commit();
      if (g < kLag) continue;
      if (g > kLag && c.j == 0) {   // a new item: its queries, once the last one's S are done
        if (!all_alive(wait(&S.q_empty, (n_q - 1) & 1, A.status, &S.abort_flag))) break;
        queries(c);
      }
      cp_wait_group<kLag>();
      const int s = (g - kLag) % kKeyStages;
      auto score = [&](int i) -> float& { return S.key[s][0][kQ ? 4 * ((lane + 32 * i) >> 1) + (lane & 1) : lane + 32 * i]; };
      const float big = fmaxf(fmaxf(fabsf(score(0)), fabsf(score(1))), fmaxf(fabsf(score(2)), fabsf(score(3))));
      if constexpr (kQ) {
        // The value scale v joins the logit as log2 v (see the softmax); where it is 0 all codes
        // are, and any v small enough not to lead will do.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = lane + 32 * i;
          const float v = S.key[s][2][j], vs = v == 0.f ? 0x1p-40f : v;
          S.key[s][2][j] = __log2f(vs);
          S.key[s][3][j] = __frcp_rn(vs);
        }
      }
      if (big > tg::kMostScore)
        for (int i = 0; i < 4; ++i) score(i) = tg::held(score(i));
      tg::mbar_arrive(&S.b_full[s]);
      c.advance(A, Q);
    }
    cp_wait_all();
    if (S.abort_flag && n_q > 0 && lane == 0)
      wait(&S.q_full, (n_q - 1) & 1, A.status, nullptr);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc<kQ>(kBM, kJob, false);
      constexpr uint32_t idesc_o = idesc<kQ>(kBM, DH, true);
      // descriptors of the first tiles; others by their distance in 16 bytes (14 bits hold them all)
      const uint64_t desc_q = tg::smem_desc_sw128(tg::smem_u32(S.q[0][0]), 16, 1024);
      const uint64_t desc_k = tg::smem_desc_sw128(tg::smem_u32(S.k[0][0]), 16, 1024);
      const uint64_t desc_v = tg::smem_desc_sw128(tg::smem_u32(S.v[0][0]), kHalfBytes, 1024);
      bool alive = true;
      int g0 = 0, jobs[2] = {}, items[2] = {};   // of either side, before this item
#pragma unroll 1
      for (int seg = 0; g0 < n && alive; ++seg) {
        // Job k of a side is half k & 1 of unit k / 2, of one row tile: half `side` of unit k. The
        // last unit may have no second half.
        const int nt = c.run(), sh = c.two ? 1 : 0;
        const int last_keys = min(kBN, c.len - (c.j + nt - 1) * kBN), no_half = last_keys <= kJob ? 1 : 0;
        const int n0 = c.two ? 2 * nt - no_half : nt, n1 = c.two ? n0 : nt - no_half;
        alive = wait(kQ ? &S.q_ready : &S.q_full, seg & 1, A.status, &S.abort_flag);
#pragma unroll 1
        for (int k = -2; k < n0 && alive; ++k) {
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const int nj = side ? n1 : n0;
            if (k >= 0 && k < nj && alive) {
              const int u = k >> sh, half = sh ? k & 1 : side, g = g0 + u, s = g % C::kV, job = jobs[side] + k;
              alive = wait(&S.p_full[side][job & 1], (job >> 1) & 1, A.status, &S.abort_flag) &&
                      wait(&S.v_full[s], (g / C::kV) & 1, A.status, &S.abort_flag);
              if (alive && k == 0 && items[side] > 0)   // the side's O of the item before has been read
                alive = wait(&S.o_free[side], (items[side] - 1) & 1, A.status, &S.abort_flag);
              if (!alive) break;
              tg::tc_fence_after();
              const uint64_t v0 = desc_v + ((s * kTileBytes + half * kJob * 128) >> 4);
              const uint32_t p0 = tmem + 128u * side + 64u * (job & 1), o = tmem + kColO + 128u * side;
              // rows of V behind the last are not set, but for those up to a multiple of 16
              const int steps = u == nt - 1 ? (min(kJob, last_keys - half * kJob) + 15) / 16 : kJob / 16;
#pragma unroll
              for (int kk = 0; kk < kJob / 16; ++kk)
                if (kk < steps)
                  tg::mma_bf16_ts(o, p0 + kk * 8, v0 + (kk * 16 * 128 >> 4), idesc_o, kk > 0 ? 1 : k > 0);
              tg::mma_commit(&S.o_done[side][job & 1]);
              // no other job reads this V
              if (sh ? side == 1 && (half == 1 || k == nj - 1) : side == 1 || k >= n1) tg::mma_commit(&S.v_empty[s]);
            }
            const int q = k + 2;
            if (q < nj && alive) {
              const int u = q >> sh, half = sh ? q & 1 : side, g = g0 + u, s = g % C::kK, job = jobs[side] + q;
              alive = wait(&S.k_full[s], (g / C::kK) & 1, A.status, &S.abort_flag);
              if (!alive) break;
              tg::tc_fence_after();
              const uint64_t k0 = desc_k + ((s * kTileBytes + half * kJob * 128) >> 4);
              const uint32_t d = tmem + 128u * side + 64u * (job & 1);
#pragma unroll
              for (int kk = 0; kk < DH / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
                tg::mma_bf16_ss(d, desc_q + ((side * kTileBytes) >> 4) + off, k0 + off, idesc_s, kk != 0);
              }
              tg::mma_commit(&S.s_full[side][job & 1]);
              if (sh ? side == 1 && (half == 1 || q == nj - 1) : side == 1 || q >= n1) tg::mma_commit(&S.k_empty[s]);
            }
          }
          if (alive && k + 3 == n0) tg::mma_commit(&S.q_empty);   // every S of the item issued
        }
        jobs[0] += n0;
        jobs[1] += n1;
        items[0] += 1;
        items[1] += n1 > 0;
        g0 += nt;
        c.advance(A, Q, nt);
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + 2 * kSideWarps) {
    // ---------------- softmax: one warp per 16 rows ----------------
    // 16x256b TMEM loads: thread l holds rows ra = l/4 and rb = ra + 8 of the warp's 16
    // at columns 8i + 2(l%4) + {0, 1}, so a row's keys sit in one quad of threads.
    const int side = (warp - 4) / kSideWarps, w8 = (warp - 4) % kSideWarps;
    const int row0 = (w8 & 3) * 32 + (w8 >> 2) * 16;
    if (row0 < rows) {
      const int r2[2] = {row0 + (lane >> 2), row0 + (lane >> 2) + 8};
      const int cq = 2 * (lane & 3);
      const uint32_t s0 = tmem + (static_cast<uint32_t>(row0) << 16) + 128u * side, obuf = s0 + kColO;
      float ch[2] = {}, gh[2] = {}, l[2] = {}, nm[2] = {}, most[2] = {};
      int seg = 0, jobs = 0, item_jobs = 0;   // jobs of this side
      bool first = true, alive = true;
#pragma unroll 1
      for (int g = 0; g < n; ++g) {
        if (first) {   // a new item
          float up[2] = {1.f, 1.f};
          if constexpr (kQ) {
            // The queries to fp16, two lanes a row: the row is multiplied by the power of two that
            // brings its largest value (exponent field x) to [2^8, 2^9), so that values down to
            // 2^-22 of it stay exact; the inverse joins the row's factor.
            alive = wait(&S.q_full, seg & 1, A.status, &S.abort_flag);
            if (!all_alive(alive)) break;
            constexpr int kPer = DH / 16;   // 16-byte columns a lane
            const int row = row0 + (lane >> 1);
            uint8_t* q = S.q[side][0] + row * 128 + (DH == 128 ? (lane & 1) * kHalfBytes : 0);
            const int c0 = DH == 128 ? 0 : 4 * (lane & 1);
            uint32_t mx = 0;
#pragma unroll 4
            for (int k = 0; k < kPer; ++k) {
              const uint4 x = *reinterpret_cast<const uint4*>(q + (((c0 + k) ^ (row & 7)) << 4));
              mx = tg::max_u16x2(mx, tg::max_u16x2(tg::max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                                   tg::max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
            }
            mx = tg::max_u16x2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            const int xp = max(static_cast<int>(max(mx >> 16, mx & 0xFFFFu) >> 7), 9);
            const float down = __int_as_float((262 - xp) << 23), inv = __int_as_float((xp - 8) << 23);
#pragma unroll 4
            for (int k = 0; k < kPer; ++k) {
              uint4* at = reinterpret_cast<uint4*>(q + (((c0 + k) ^ (row & 7)) << 4));
              const uint4 x = *at;
              *at = make_uint4(tg::bf16x2_to_f16x2(x.x, down), tg::bf16x2_to_f16x2(x.y, down),
                               tg::bf16x2_to_f16x2(x.z, down), tg::bf16x2_to_f16x2(x.w, down));
            }
            up[0] = __shfl_sync(0xFFFFFFFFu, inv, 2 * (lane >> 2));
            up[1] = __shfl_sync(0xFFFFFFFFu, inv, 2 * (lane >> 2) + 16);
            tg::fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) tg::mbar_arrive(&S.q_ready);
          }
          // rows behind the last hold anything: with factors of zero they leave the reference alone
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int hq = c.kvh * A.group + r2[e] - tg::token_of(A, r2[e]) * A.group;
            ch[e] = r2[e] < rows ? kLog2e / (sqrtf(static_cast<float>(DH)) * A.tau[hq]) * up[e] : 0.f;
            gh[e] = r2[e] < rows ? A.gain[hq] * kLog2e : 0.f;
            most[e] = -INFINITY;   // nothing seen: logits as they are, and any of them moves the reference
            nm[e] = l[e] = 0.f;
          }
          item_jobs = 0;
        }
        const int s = g % kKeyStages;
        alive = wait(&S.b_full[s], (g / kKeyStages) & 1, A.status, &S.abort_flag);
        const int nv = c.keys();
#pragma unroll 1
        for (int half = c.two ? 0 : side; alive && kJob * half < nv; ++half) {
          const uint32_t sbuf = s0 + 64u * (jobs & 1);
          alive = wait(&S.s_full[side][jobs & 1], (jobs >> 1) & 1, A.status, &S.abort_flag);
          if (!all_alive(alive)) { alive = false; break; }
          tg::tc_fence_after();
          const int nh = nv - kJob * half;
          const float* key = S.key[s][0] + kJob * half + cq;
          float z[32];
          {
            uint32_t u[32];
            tg::tmem_ld_16x256b_x8(sbuf, u);
            tg::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x[4] = {__uint_as_float(u[4 * i]), __uint_as_float(u[4 * i + 1]),
                            __uint_as_float(u[4 * i + 2]), __uint_as_float(u[4 * i + 3])};
              float2 sk, lv = {};
              if constexpr (kQ) {
                const float4 both = *reinterpret_cast<const float4*>(S.key[s][0] + 2 * (kJob * half + cq + 8 * i));
                sk = make_float2(both.x, both.y);
                lv = *reinterpret_cast<const float2*>(key + 2 * kBN + 8 * i);
                fmul2(x[0], x[1], x[0], x[1], both.z, both.w);
                fmul2(x[2], x[3], x[2], x[3], both.z, both.w);
              } else {
                sk = *reinterpret_cast<const float2*>(key + 8 * i);
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float b0, b1;
                if constexpr (kQ) ffma2(b0, b1, gh[e], gh[e], sk.x, sk.y, lv.x, lv.y);
                else fmul2(b0, b1, gh[e], gh[e], sk.x, sk.y);
                ffma2(z[4 * i + 2 * e], z[4 * i + 2 * e + 1], x[2 * e], x[2 * e + 1], ch[e], ch[e], b0, b1);
              }
            }
          }
          if (nh < kJob) {   // keys that are not there
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int f = 0; f < 2; ++f)
                if (8 * i + cq + f >= nh) z[4 * i + f] = z[4 * i + 2 + f] = -INFINITY;
          }
          float mx[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t0 = fmaxf(z[2 * e], z[2 * e + 1]), t1 = fmaxf(z[4 + 2 * e], z[5 + 2 * e]);
#pragma unroll
            for (int i = 2; i < 8; i += 2) {
              t0 = fmax3(t0, z[4 * i + 2 * e], z[4 * i + 2 * e + 1]);
              t1 = fmax3(t1, z[4 * i + 4 + 2 * e], z[4 * i + 5 + 2 * e]);
            }
            mx[e] = fmaxf(t0, t1);
          }
          // A row's reference is a whole number at or above its largest logit (fp16 weights: 6
          // below that, to keep small ones exact) when it is set, so that moving it scales by an
          // exact power of two; it moves when a logit exceeds it by 2^8 more, so that bf16 weights
          // stay below 2^8 and fp16 ones below 2^14. It is taken off logits that are rounded
          // already: of the largest nothing but the lift is left, however large they are.
          if (__any_sync(0xFFFFFFFFu, mx[0] + nm[0] > most[0] || mx[1] + nm[1] > most[1])) {
            constexpr float kLift = kQ ? 6.f : 0.f;
            float alpha[2] = {1.f, 1.f};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 1));
              mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 2));
              if (mx[e] + nm[e] > most[e]) {
                const float to = kLift - ceilf(mx[e]);
                alpha[e] = most[e] == -INFINITY ? 0.f : tg::exp2_approx(to - nm[e]);   // 0 where nothing was seen
                nm[e] = to;
                most[e] = kLift + tg::kRescaleThreshold;
                l[e] *= alpha[e];
              }
            }
            if (item_jobs > 0) {   // once O holds the jobs before
              alive = wait(&S.o_done[side][(jobs - 1) & 1], ((jobs - 1) >> 1) & 1, A.status, &S.abort_flag);
              __syncwarp();
              tg::tc_fence_after();
#pragma unroll 1
              for (int h = 0; h < DH / 16; ++h) {
                uint32_t o[8];
                tmem_ld_16x256b_x2(obuf + 16u * h, o);
                tg::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[(i >> 1) & 1]);
                tmem_st_16x256b_x2(obuf + 16u * h, o);
              }
            }
          }
          // Weights 2^z. Codes: log2 v is part of z, so these are what the codes are multiplied
          // by and the reference follows their largest; the row sum takes them in fp32, divided by
          // v. bf16: the row sum adds the rounded weights, so that a key which dominates its row
          // gives its value exactly.
          uint32_t pk[16];
          float sum[2][2] = {};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float2 iv = {};
            if constexpr (kQ) iv = *reinterpret_cast<const float2*>(key + 3 * kBN + 8 * i);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float p0, p1;
              fadd2(p0, p1, z[4 * i + 2 * e], z[4 * i + 2 * e + 1], nm[e], nm[e]);
              p0 = tg::exp2_approx(p0), p1 = tg::exp2_approx(p1);
              if constexpr (kQ) {
                pk[2 * i + e] = tg::pack_f16x2(p0, p1);
                ffma2(sum[e][0], sum[e][1], p0, p1, iv.x, iv.y, sum[e][0], sum[e][1]);
              } else {
                pk[2 * i + e] = tg::pack_bf16x2(p0, p1);
                add_bf16_lo(sum[e][0], pk[2 * i + e]);
                add_bf16_hi(sum[e][1], pk[2 * i + e]);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) l[e] += sum[e][0] + sum[e][1];
          tmem_st_16x128b_x8(sbuf, pk);   // P over S, which is read
          tg::tmem_st_wait();
          tg::tc_fence_before();
          __syncwarp();
          if (lane == 0) tg::mbar_arrive(&S.p_full[side][jobs & 1]);
          ++jobs;
          ++item_jobs;
          if (!c.two) break;
        }
        if (!all_alive(alive)) { alive = false; break; }
        __syncwarp();
        if (lane == 0) tg::mbar_arrive(&S.b_empty[s]);   // this warp is done with the keys' data
        first = c.run() == 1;   // the last unit of its item here: O is complete after the last PV
        if (first) {
          // CTA c and item i (numbered over all sequences): slot c + i grows along the units
          const int item = (c.b * A.n_hkv + c.kvh) * tg::row_pairs(A, A.n_draft) + c.pair;
          const int64_t slot = (static_cast<int64_t>(blockIdx.x + item) * 2 + side) * rows;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
            l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
          }
          if (item_jobs > 0) {
            alive = wait(&S.o_done[side][(jobs - 1) & 1], ((jobs - 1) >> 1) & 1, A.status, &S.abort_flag);
            if (!all_alive(alive)) { alive = false; break; }
            tg::tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < DH / 16; ++h) {   // columns cq and cq + 1 of each 8
              uint32_t o[8];
              tmem_ld_16x256b_x2(obuf + 16u * h, o);
              tg::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (r2[e] < rows) {
                  float* p = A.part + (slot + r2[e]) * DH + 16 * h + cq;
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint2*>(p + 8 * i) = make_uint2(o[4 * i + 2 * e], o[4 * i + 2 * e + 1]);
                }
              __syncwarp();
            }
            tg::tc_fence_before();
            __syncwarp();
            if (lane == 0) tg::mbar_arrive(&S.o_free[side]);   // O may be overwritten
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)   // without a job: a sum of nothing, whose O is not read
            if ((lane & 3) == 0 && r2[e] < rows)
              *reinterpret_cast<float2*>(tg::part_ml(A, rows, DH) + (slot + r2[e]) * 2) =
                  make_float2(most[e] == -INFINITY ? most[e] : -nm[e], l[e]);
          ++seg;
        }
        c.advance(A, Q);
      }
    }
  } else if (kQ && warp >= 4 + 2 * kSideWarps) {
    // ---------------- codes to operand tiles, 32 rows a warp ----------------
    constexpr bool kE4m3 = kType == TG_E4M3;
    const int cw = warp - 4 - 2 * kSideWarps;
    // Eight lanes take one 16-code column of eight rows, so that reads of the swizzled raw
    // tile and stores to the swizzled operand tile both fall into different banks.
    constexpr int kC16 = DH / 16;                          // 16-code columns of a row
    constexpr int kRows = kBN / kConvWarps;                // rows of a warp
    constexpr int kPasses = kRows * kC16 / 32;
    const int rl = lane & 7, cl = lane >> 3;               // row of eight, column of four
    int gk = 0, gv = 0, keys = 0, last_keys = 0;
#pragma unroll 1
    for (int r = 0; r < 2 * n; ++r) {
      const bool val = value_turn(r, n);
      if (!val) {
        last_keys = keys;
        keys = c.keys();
        c.advance(A, Q);
      }
      const int g = val ? gv++ : gk++, n_st = val ? C::kV : C::kK, s = g % n_st;
      const int nv = val && r < 2 * n - 1 ? last_keys : keys;
      uint64_t* full = val ? &S.v_full[s % C::kV] : &S.k_full[s % C::kK];
      uint64_t* empty = val ? &S.v_empty[s % C::kV] : &S.k_empty[s % C::kK];
      uint8_t* dst = val ? S.v[s % C::kV][0] : S.k[s % C::kK][0];
      const int rs = r % C::kRaw;
      if (!all_alive(wait(&S.raw_full[rs], (r / C::kRaw) & 1, A.status, &S.abort_flag))) break;
      const uint8_t* src = S.raw[rs];
      uint4 x[kPasses];
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int rr = kRows * cw + 8 * (p / (kC16 / 4)) + rl, cc = cl + 4 * (p % (kC16 / 4));
        x[p] = *reinterpret_cast<const uint4*>(src + rr * DH + ((DH == 128 ? cc ^ rl : cc ^ ((rl >> 1) & 3)) << 4));
        if (val && rr >= nv) x[p] = make_uint4(0, 0, 0, 0);   // rows behind the end weigh 0
      }
      if (g >= n_st && !all_alive(wait(empty, ((g / n_st) - 1) & 1, A.status, &S.abort_flag))) break;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int rr = kRows * cw + 8 * (p / (kC16 / 4)) + rl, cc = cl + 4 * (p % (kC16 / 4));
        const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
        uint32_t y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tg::widen4<kE4m3>(w[e] ^ (kE4m3 ? 0u : 0x80808080u), y[2 * e], y[2 * e + 1]);
        *reinterpret_cast<uint4*>(dst + tile_off(rr, 2 * cc)) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(dst + tile_off(rr, 2 * cc + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
      }
      // The raw tile is given back only now: its loads have all arrived and are ordered before
      // the next copy into it. Given back when they were only under way, it was overwritten
      // under one about once in 200 calls.
      tg::fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        tg::mbar_arrive(&S.raw_empty[rs]);
        tg::mbar_arrive(full);
      }
    }
  }
  tg::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tg::tc_fence_after();
    tg::tmem_dealloc(tmem, kTmemCols);
  }
}

// Adds up what the CTAs left of every output row and brings in the drafted rows that its
// token sees, key by key, so that what it does not see is not even read. Eight lanes are a
// stream with its own running maximum, sum and O (16 or 8 dims a lane); the 4 kW streams of
// a row take its partials (of the CTAs c0 .. c1 that share its item, in order: those of a
// row tile's side, or of all kw parts of its keys) and then its drafted rows in turn, two in
// flight at a time, and are joined in a fixed order. CTA c's partial of item i (numbered over
// all sequences) is in slot c + i.
template <int DH, int kW>
__global__ void __launch_bounds__(128) tree_combine_kernel(const __grid_constant__ TreeArgs A) {
  constexpr int kC = DH / 64;           // 8-dim pieces of a lane: dims 64 p + 8 (lane % 8) ..
  constexpr int kE = 8 * kC;
  constexpr int kRows = 4 / kW;         // rows of a block, neighbouring heads
  constexpr int kNs = 4 * kW;           // streams of a row
  constexpr int kD = 2;
  __shared__ float red[4][DH + 2];
  tg::pdl_launch_dependents();
  tg::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i8 = lane & 7;
  const int stream = (warp % kW) * 4 + (lane >> 3);
  const int hq = blockIdx.x * kRows + warp / kW, t = blockIdx.y, b = blockIdx.z;
  const bool mine = hq < A.n_hq;        // the last block's last warps may have no row
  const int hr = mine ? hq : 0, kvh = hr / A.group;
  // what does not wait for anything else is asked for at once
  const int64_t bt = static_cast<int64_t>(b) * A.n_draft + t;
  const int W = A.base[A.batch], first0 = A.base[b];
  const int2 sl = tg::seq_lens(A, b, false);
  uint64_t see = static_cast<uint64_t>(A.mask[bt]);
  uint4 qw[kC];
#pragma unroll
  for (int p = 0; p < kC; ++p) qw[p] = *reinterpret_cast<const uint4*>(A.q + (bt * A.n_hq + hr) * DH + 64 * p + 8 * i8);
  const float tau = A.tau[hr], gain = A.gain[hr];
  if (t >= sl.y) return;
  auto widen = [](const uint4& h, float* f) {
    const uint32_t u[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = bf16_lo(u[e]);
      f[2 * e + 1] = bf16_hi(u[e]);
    }
  };
  // the stream's drafted rows: visible ones stream, stream + kNs, ..
  if (sl.y < 64) see &= (1ull << sl.y) - 1;
  int left = (__popcll(see) + kNs - 1) / kNs;   // the longest stream's rows
  for (int i = 0; i < stream; ++i) see &= see - 1;
  uint4 kh[kD][kC] = {}, vh[kD][kC] = {};
  float sd[kD] = {};
  bool has[kD];
  auto drafted = [&]() {
#pragma unroll
    for (int d = 0; d < kD; ++d) {
      has[d] = see != 0;
      if (!has[d]) continue;
      const int64_t at = static_cast<int64_t>(b) * A.n_draft + __ffsll(static_cast<long long>(see)) - 1;
#pragma unroll
      for (int p = 0; p < kC; ++p) {
        kh[d][p] = *reinterpret_cast<const uint4*>(A.kd + (at * A.n_hkv + kvh) * DH + 64 * p + 8 * i8);
        vh[d][p] = *reinterpret_cast<const uint4*>(A.vd + (at * A.n_hkv + kvh) * DH + 64 * p + 8 * i8);
      }
      sd[d] = tg::held(A.sd[at]);
#pragma unroll
      for (int i = 0; i < kNs; ++i) see &= see - 1;
    }
  };
  drafted();
  float M = -INFINITY, L = 0.f, acc[kE] = {};
  const int nt = tg::key_units(A, sl.x);
  if (nt > 0) {
    const tg::Shares share(A, W);
    const int group = kvh / A.hw, hd = kvh - group * A.hw, mt = t / A.tm;
    const int row = (t - mt * A.tm) * A.group + hr - kvh * A.group, rows = A.group * A.tm;
    const bool two = (mt | 1) < tg::row_tiles(A, sl.y);   // a side of its own
    const int first = first0 + (group * tg::row_pairs(A, sl.y) + mt / 2) * nt;
    const int c0 = share.cta_of(first), c1 = share.cta_of(first + nt - 1);
    const int slot0 = c0 + (b * tg::head_groups(A) + group) * tg::row_pairs(A, A.n_draft) + mt / 2;
    const int parts = A.hw * A.kw, kw = two ? 1 : A.kw, part0 = hd * A.kw + (two ? mt & 1 : 0);
    const int n = (c1 - c0 + 1) * kw;
    const float* ml = tg::part_ml(A, rows, DH);
#pragma unroll 1
    for (int i0 = stream; i0 < n; i0 += kD * kNs) {
      float2 v[kD];
      float4 x[kD][2 * kC];
#pragma unroll
      for (int k = 0; k < kD; ++k) {
        const int i = i0 + kNs * k, ci = kw == 1 ? i : i / kw;
        const int64_t at = (static_cast<int64_t>(slot0 + ci) * parts + part0 + (i - ci * kw)) * rows + row;
        v[k] = make_float2(-INFINITY, 0.f);
        if (i >= n) continue;
        v[k] = *reinterpret_cast<const float2*>(ml + at * 2);
#pragma unroll
        for (int p = 0; p < 2 * kC; ++p)
          x[k][p] = *reinterpret_cast<const float4*>(A.part + at * DH + 64 * (p >> 1) + 8 * i8 + 4 * (p & 1));
      }
      float mb = M;
#pragma unroll
      for (int k = 0; k < kD; ++k) mb = fmaxf(mb, v[k].x);
      const float base = mb == -INFINITY ? 0.f : mb, scale = tg::exp2_approx(M - base);
      M = mb;
      L *= scale;
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[e] *= scale;
#pragma unroll
      for (int k = 0; k < kD; ++k) {
        const float wk = tg::exp2_approx(v[k].x - base);
        if (v[k].y == 0.f) continue;   // a part without keys has no O
        L = fmaf(wk, v[k].y, L);
#pragma unroll
        for (int p = 0; p < 2 * kC; ++p) {
          acc[4 * p] = fmaf(wk, x[k][p].x, acc[4 * p]);
          acc[4 * p + 1] = fmaf(wk, x[k][p].y, acc[4 * p + 1]);
          acc[4 * p + 2] = fmaf(wk, x[k][p].z, acc[4 * p + 2]);
          acc[4 * p + 3] = fmaf(wk, x[k][p].w, acc[4 * p + 3]);
        }
      }
    }
    __syncwarp();
  }
  const float ch = kLog2e / (sqrtf(static_cast<float>(DH)) * tau), gh = gain * kLog2e;
  float qf[kE];
#pragma unroll
  for (int p = 0; p < kC; ++p) widen(qw[p], qf + 8 * p);
#pragma unroll 1
  for (; left > 0; left -= kD) {   // all streams of the warp together: their shuffles
    float z[kD], mn = M;
    uint4 vk[kD][kC];
#pragma unroll
    for (int d = 0; d < kD; ++d) {
      z[d] = 0.f;
#pragma unroll
      for (int p = 0; p < kC; ++p) {
        float kf[8];
        widen(kh[d][p], kf);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[d] = fmaf(qf[8 * p + e], kf[e], z[d]);
        vk[d][p] = vh[d][p];
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) z[d] += __shfl_xor_sync(0xFFFFFFFFu, z[d], o);
      z[d] = has[d] ? fmaf(z[d], ch, gh * sd[d]) : -INFINITY;
      mn = fmaxf(mn, z[d]);
    }
    drafted();
    const float base = mn == -INFINITY ? 0.f : mn, scale = tg::exp2_approx(M - base);
    M = mn;
    L *= scale;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] *= scale;
#pragma unroll
    for (int d = 0; d < kD; ++d) {
      if (z[d] == -INFINITY) continue;   // a weight of zero: its values do not count, whatever they are
      const float p = tg::exp2_approx(z[d] - base);
      L += p;
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        float vf[8];
        widen(vk[d][i], vf);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[8 * i + e] = fmaf(p, vf[e], acc[8 * i + e]);
      }
    }
    __syncwarp();
  }
  // the warp's streams, then its warps
  float mw = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, 8));
  mw = fmaxf(mw, __shfl_xor_sync(0xFFFFFFFFu, mw, 16));
  const float down = tg::exp2_approx(M - (mw == -INFINITY ? 0.f : mw));
  L *= down;
  L += __shfl_xor_sync(0xFFFFFFFFu, L, 8);
  L += __shfl_xor_sync(0xFFFFFFFFu, L, 16);
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    acc[e] *= down;
    acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], 8);
    acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], 16);
  }
  const int64_t at = bt * A.n_hq + hr;
  if constexpr (kW == 1) {
    const float inv = L == 0.f ? 0.f : 1.f / L;   // nothing seen: zeros
    if (!mine || lane >= 8 || !tg::in_bounds(at, static_cast<int64_t>(A.batch) * A.n_draft * A.n_hq, A.status)) return;
#pragma unroll
    for (int p = 0; p < kC; ++p) {
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = tg::pack_bf16x2(acc[8 * p + 2 * e] * inv, acc[8 * p + 2 * e + 1] * inv);
      *reinterpret_cast<uint4*>(A.out + at * DH + 64 * p + 8 * i8) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  } else {
    if (lane < 8) {
#pragma unroll
      for (int e = 0; e < kE; ++e) red[warp][64 * (e >> 3) + 8 * i8 + (e & 7)] = acc[e];
    }
    if (lane == 0) {
      red[warp][DH] = mw;
      red[warp][DH + 1] = L;
    }
    __syncthreads();
    const int d = threadIdx.x;
    if (d >= DH) return;
    float Mx = -INFINITY, Lx = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w) Mx = fmaxf(Mx, red[w][DH]);
    const float base = Mx == -INFINITY ? 0.f : Mx;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const float f = tg::exp2_approx(red[w][DH] - base);
      Lx = fmaf(f, red[w][DH + 1], Lx);
      y = fmaf(f, red[w][d], y);
    }
    if (!tg::in_bounds(at, static_cast<int64_t>(A.batch) * A.n_draft * A.n_hq, A.status)) return;
    A.out[at * DH + d] = __float2bfloat16_rn(y * (Lx == 0.f ? 0.f : 1.f / Lx));   // nothing seen: zeros
  }
}

// Fewer units a CTA than this cost more in partials than the CTAs are worth. One single token
// / eight tokens of two heads over 1868 rows: 12.3 / 17.9 us with one, 11.6 / 15.9 us with two,
// 14.2 / 19.1 us with four.
constexpr int kMinUnits = 2;

// Warps a row in the combining kernel: four where there are few rows, or not many and each
// with many partials; one where the rows fill the machine anyhow. With one and with four:
// 128 rows 14.1 and 12.9 us, 1024 rows of 28 partials 105 and 72 us, 1024 rows of 3 partials
// 19.4 and 21.6 us, 1664 rows of 7 partials 57.2 and 61.9 us, 4096 rows 27.9 and 44.0 us.
bool four_warps(int64_t rows, int64_t partials) { return rows <= 512 || (rows <= 2048 && partials > 16); }

// How a call is laid out: which kernel, tokens per row tile, units, CTAs and the
// workspace's two parts.
struct Plan {
  bool few;   // tree_rows_kernel
  int tm, unit, hw, kw, n_cta;
  int64_t units, slots;
  size_t base_bytes, bytes;
};
Plan plan(int batch, int n_draft, int max_len, int n_hq, int n_hkv, int head_dim, bool codes) {
  Plan p;
  const int group = n_hq / n_hkv;
  const int most_tm = kBM / group, tiles = (n_draft + most_tm - 1) / most_tm;
  p.tm = (n_draft + tiles - 1) / tiles;   // tiles alike
  const int rows = group * p.tm;
  // Which kernel (this one and tree_rows.cu): codes, 8 x 10721 rows of eight heads: 2 rows a KV
  // head (32 x 1868) 79 and 38 us, 16 rows 104 and 72 us, 26 rows 105 and 113 us (head dim 64: 62
  // and 33 us, 77 and 62 us, 26 rows not measured); a bf16 cache: 2 rows 52.6 and 52.8 us, 16 rows
  // (one of 1868) 12.9 and 14.4 us, 26 rows 61 and 67 us. The figures of tree_rows.cu beyond 16
  // rows and over bf16 are those of forms that it no longer has.
  p.few = codes && rows <= tg::kTreeRowsMax;
  const int warps = tg::tree_rows_warps(rows);
  p.hw = p.few ? (n_hkv < warps ? n_hkv : warps) : 1;
  p.kw = p.few ? warps / p.hw : 2;
  p.unit = p.few ? 16 * p.kw : kBN;
  auto units_of = [&](int64_t keys) { return (keys + p.unit - 1) / p.unit; };
  const int64_t items = static_cast<int64_t>(batch) * ((n_hkv + p.hw - 1) / p.hw) * ((tiles + 1) / 2);
  p.units = items * units_of(max_len);
  const int64_t most = p.few ? tg::tree_rows_ctas(rows) : kMaxCtas;
  // few rows: no fewer than kMinUnits units a CTA, since every CTA leaves a partial
  const int64_t want = p.few ? (p.units + kMinUnits - 1) / kMinUnits : p.units;
  p.n_cta = static_cast<int>(want < 1 ? 1 : want < most ? want : most);
  p.slots = p.n_cta + items;
  p.base_bytes = (static_cast<size_t>(batch) + 1) * sizeof(int32_t);
  p.base_bytes = (p.base_bytes + 255) / 256 * 256;
  p.bytes = p.base_bytes +
            static_cast<size_t>(p.slots) * p.hw * p.kw * rows * (head_dim + 2) * sizeof(float);
  return p;
}

template <int DH>
tg_status launch_combine(const TreeArgs& a, tg_status r, cudaStream_t st) {
  if (r != TG_OK) return r;
  const int64_t rows = static_cast<int64_t>(a.batch) * a.n_draft * a.n_hq;
  if (four_warps(rows, a.n_cta / (a.slots - a.n_cta) * a.kw))
    return tg::launch(tree_combine_kernel<DH, 4>, dim3(a.n_hq, a.n_draft, a.batch), dim3(128), 0, st, 0, a);
  return tg::launch(tree_combine_kernel<DH, 1>, dim3((a.n_hq + 3) / 4, a.n_draft, a.batch), dim3(128), 0, st, 0, a);
}

template <int DH, int kType>
tg_status launch_tree(const TreeArgs& a, cudaStream_t st) {
  constexpr bool kQ = kType != TG_BF16;
  using C = Cfg<DH, kQ>;
  CUtensorMap tq, tk, tv;
  const uint64_t qdims[3] = {DH, static_cast<uint64_t>(a.n_hq), static_cast<uint64_t>(a.batch) * a.n_draft};
  const uint64_t qstr[2] = {DH * 2, static_cast<uint64_t>(a.n_hq) * DH * 2};
  const uint32_t qbox[3] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(a.tm)};
  if (!tg::encode_tmap(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, qdims, qstr, qbox,
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tg::tree_cache_map(a, a.kc, DH, kQ, kBN, 1, &tk) || !tg::tree_cache_map(a, a.vc, DH, kQ, kBN, 1, &tv))
    return TG_ERR_CUDA;
  constexpr int smem = sizeof(TreeSmem<DH, kQ>) + 1024;
  static_assert(smem <= 232448, "the shared memory of one SM");
  if (!tg::ensure_smem(reinterpret_cast<const void*>(tree_attn_kernel<DH, kType>), smem)) return TG_ERR_CUDA;
  return launch_combine<DH>(
      a, tg::launch(tree_attn_kernel<DH, kType>, dim3(a.n_cta), dim3(C::kThreads), smem, st, 0, tq, tk, tv, a), st);
}

}  // namespace

extern "C" size_t tg_tree_attention_workspace_size(int batch, int n_draft, int max_len, int n_hq,
                                                   int n_hkv, int head_dim) {
  if (batch <= 0 || n_draft <= 0 || max_len < 0 || n_hkv <= 0 || n_hq < n_hkv || n_hq / n_hkv > kBM ||
      head_dim <= 0)
    return 0;
  // for either kind of cache
  const size_t a = plan(batch, n_draft, max_len, n_hq, n_hkv, head_dim, false).bytes;
  const size_t b = plan(batch, n_draft, max_len, n_hq, n_hkv, head_dim, true).bytes;
  return a > b ? a : b;
}

extern "C" tg_status tg_tree_attention(
    const void* q, const void* k_draft, const void* v_draft, const float* s_draft,
    const int64_t* tree_mask, const int32_t* draft_len, int batch, int n_draft,
    const void* k_cache, const void* v_cache, tg_dtype cache_dtype, const float* k_scale,
    const float* v_scale, const float* s_cache, const int32_t* cache_len, int cap, int max_len,
    int n_hq, int n_hkv, int head_dim, const float* gain, const float* tau, void* out,
    void* workspace, size_t workspace_bytes, tg_stream_t stream) {
  tg::NvtxRange nvtx_range("tg_tree_attention");
  if (batch < 0 || n_draft < 0 || cap <= 0 || max_len < 0 || n_hq <= 0 || n_hkv <= 0 ||
      head_dim <= 0 || max_len > cap || n_hq % n_hkv != 0)
    return TG_ERR_INVALID_ARG;
  if (cache_dtype != TG_BF16 && cache_dtype != TG_I8 && cache_dtype != TG_E4M3)
    return TG_ERR_UNSUPPORTED;
  if (batch == 0 || n_draft == 0) return TG_OK;
  if (!q || !k_draft || !v_draft || !s_draft || !tree_mask || !k_cache || !v_cache || !s_cache ||
      !cache_len || !gain || !tau || !out)
    return TG_ERR_INVALID_ARG;
  const bool quantised = cache_dtype != TG_BF16;
  if (quantised ? !k_scale || !v_scale : k_scale || v_scale) return TG_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || n_draft > kMaxDraft || n_hq / n_hkv > kBM ||
      batch > tg::kTreeMaxBatch || n_hkv > 1024 || static_cast<int64_t>(batch) * cap > INT32_MAX - kBN)
    return TG_ERR_UNSUPPORTED;
  if (!tg::aligned16(q) || !tg::aligned16(k_draft) || !tg::aligned16(v_draft) ||
      !tg::aligned16(k_cache) || !tg::aligned16(v_cache) || !tg::aligned16(out))
    return TG_ERR_MISALIGNED;
  const Plan p = plan(batch, n_draft, max_len, n_hq, n_hkv, head_dim, quantised);
  if (p.units > INT32_MAX / 2) return TG_ERR_UNSUPPORTED;   // far more keys than a GPU holds
  if (!workspace || workspace_bytes < tg_tree_attention_workspace_size(batch, n_draft, max_len, n_hq, n_hkv, head_dim))
    return TG_ERR_WORKSPACE;
  if (!tg::aligned16(workspace)) return TG_ERR_MISALIGNED;
  TreeArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.kd = static_cast<const __nv_bfloat16*>(k_draft), a.vd = static_cast<const __nv_bfloat16*>(v_draft);
  a.sd = s_draft, a.mask = tree_mask, a.draft_len = draft_len;
  a.kc = static_cast<const uint8_t*>(k_cache), a.vc = static_cast<const uint8_t*>(v_cache);
  a.ks = k_scale, a.vs = v_scale, a.sc = s_cache, a.cache_len = cache_len;
  a.gain = gain, a.tau = tau, a.out = static_cast<__nv_bfloat16*>(out);
  a.base = static_cast<int32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.base_bytes);
  a.batch = batch, a.n_draft = n_draft, a.cap = cap, a.max_len = max_len, a.n_hq = n_hq, a.n_hkv = n_hkv;
  a.group = n_hq / n_hkv, a.group_inv = (65536 + a.group - 1) / a.group, a.tm = p.tm, a.unit = p.unit, a.hw = p.hw, a.kw = p.kw, a.n_cta = p.n_cta;
  a.slots = p.slots;
  a.status = tg::status_word();
  if (!a.status) return TG_ERR_CUDA;
  if (p.few) {
    const tg_status r = tg::launch_tree_rows(a, head_dim, cache_dtype, stream);
    return head_dim == 128 ? launch_combine<128>(a, r, stream) : launch_combine<64>(a, r, stream);
  }
  if (head_dim == 128) {
    if (cache_dtype == TG_BF16) return launch_tree<128, TG_BF16>(a, stream);
    return cache_dtype == TG_I8 ? launch_tree<128, TG_I8>(a, stream) : launch_tree<128, TG_E4M3>(a, stream);
  }
  if (cache_dtype == TG_BF16) return launch_tree<64, TG_BF16>(a, stream);
  return cache_dtype == TG_I8 ? launch_tree<64, TG_I8>(a, stream) : launch_tree<64, TG_E4M3>(a, stream);
}

// What the kernels of tg_tree_attention share: their arguments, and the split of all work
// into equal shares.
//
// Work units are pieces of `unit` cache rows. An item is a sequence's KV heads, `hw` at a
// time, and a pair of tiles of its query rows (or one tile); it has the units of its cache. All units of all items
// are numbered in a row, and every CTA takes an equal share of that row, so ragged lengths
// and few heads fill the machine alike.
#pragma once

#include "common.cuh"

namespace tg {

constexpr int kTreeMaxBatch = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMostScore = 0x1p120f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units a logit may exceed the reference by

struct TreeArgs {
  const __nv_bfloat16 *q, *kd, *vd;
  const float* sd;
  const int64_t* mask;
  const int32_t* draft_len;
  const uint8_t *kc, *vc;
  const float *ks, *vs, *sc;
  const int32_t* cache_len;
  const float *gain, *tau;
  __nv_bfloat16* out;
  int32_t* base;      // [batch + 1] first unit of each sequence (written by CTA 0)
  float* part;        // partials: [slots][hw * kw][rows][dh], then [slots][hw * kw][rows][2] (max, sum)
  int64_t slots;
  int batch, n_draft, cap, max_len, n_hq, n_hkv;
  int group, group_inv;   // query heads per KV head; ceil(2^16 / group)
  int tm;             // tokens of a row tile
  int unit;           // keys of a unit
  int hw, kw;         // KV heads of an item, and parts (warps, sides) that its keys or rows are split in
  int n_cta;
  int* status;
};

// row / group for row < 2^8: group_inv exceeds 2^16 / group by less than 1, so the product
// exceeds 2^16 row / group by less than 2^8 < 2^16 / group.
__device__ __forceinline__ int token_of(const TreeArgs& A, int row) { return (row * A.group_inv) >> 16; }

// A sequence's lengths, or no drafted tokens where they are out of range.
__device__ __forceinline__ int2 seq_lens(const TreeArgs& A, int b, bool record) {
  const int len = A.cache_len[b], dl = A.draft_len ? A.draft_len[b] : A.n_draft;
  if (len < 0 || len > A.cap || len > A.max_len || dl < 0 || dl > A.n_draft) {
    if (record) set_status(A.status, TG_ERR_DEVICE_CHECK);
    return make_int2(0, 0);
  }
  return make_int2(len, dl);
}
__device__ __forceinline__ int row_tiles(const TreeArgs& A, int dl) { return (dl + A.tm - 1) / A.tm; }
__device__ __forceinline__ int row_pairs(const TreeArgs& A, int dl) { return (row_tiles(A, dl) + 1) / 2; }
__device__ __forceinline__ int key_units(const TreeArgs& A, int keys) { return (keys + A.unit - 1) / A.unit; }
__device__ __forceinline__ int head_groups(const TreeArgs& A) { return (A.n_hkv + A.hw - 1) / A.hw; }
// Where the maxima and sums of the partials begin.
__device__ __forceinline__ float* part_ml(const TreeArgs& A, int rows, int dh) {
  return A.part + A.slots * A.hw * A.kw * rows * dh;
}

// W units over G = min(CTAs, W) CTAs: the first `more` take each + 1 units, the others
// `each`, so none is empty and every CTA between an item's first and last holds a part of
// it.
struct Shares {
  int n, each, more;
  __device__ __forceinline__ Shares(const TreeArgs& A, int W) {
    n = W < A.n_cta ? W : A.n_cta;
    each = n ? W / n : 0;
    more = n ? W - each * n : 0;
  }
  __device__ __forceinline__ int first(int cta) const { return cta >= n ? 0 : cta * each + (cta < more ? cta : more); }
  __device__ __forceinline__ int size(int cta) const { return cta >= n ? 0 : each + (cta < more); }
  __device__ __forceinline__ int cta_of(int u) const {
    const int big = more * (each + 1);
    return u < big ? u / (each + 1) : more + (u - big) / each;
  }
};

// Per sequence, in shared memory: first unit (one more: the end), cache length, drafted tokens.
struct TreeSeqs {
  int *base, *len;
  uint8_t* dl;
};

// Every sequence's lengths and first unit into shared memory (CTA 0: the units also to the
// workspace, for the second kernel); all threads of the block, with barriers. Returns the
// number of units, below 2^31 (the host sees to it).
template <int kThreads>
__device__ __forceinline__ int count_units(const TreeArgs& A, const TreeSeqs& S) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int b = tid; b < A.batch; b += kThreads) {
    const int2 l = seq_lens(A, b, blockIdx.x == 0);
    S.len[b] = l.x;
    S.dl[b] = static_cast<uint8_t>(l.y);
    S.base[b + 1] = l.y ? head_groups(A) * row_pairs(A, l.y) * key_units(A, l.x) : 0;
  }
  __syncthreads();
  if (tid < 32) {
    int carry = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < A.batch; b0 += 32) {
      int x = b0 + lane < A.batch ? S.base[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < A.batch) S.base[b0 + lane + 1] = carry + x;
      carry += __shfl_sync(0xFFFFFFFFu, x, 31);
    }
    if (lane == 0) S.base[0] = 0;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = tid; b <= A.batch; b += kThreads) A.base[b] = S.base[b];
  return S.base[A.batch];
}

// The last sequence whose first unit is at most u.
__device__ __forceinline__ int sequence_of(const TreeArgs& A, const TreeSeqs& S, int u) {
  int lo = 0, hi = A.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (S.base[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The slow side of a wait is one function: with it inlined at every site the loops of the
// kernels' roles no longer fit the instruction cache together.
__device__ __noinline__ inline bool wait_slow(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  return mbar_wait(bar, parity, status, abort);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  return mbar_try_wait(smem_u32(bar), parity) || wait_slow(bar, parity, status, abort);
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// A score as logits take it: gain * score * log2(e) of a finite score is finite too (up to gains of
// 88), so that rows which see nothing but scores of the type's lowest value still have a
// largest one. Infinities and NaN stay what they are.
__device__ __forceinline__ float held(float s) {
  return fabsf(s) > kMostScore && fabsf(s) < INFINITY ? copysignf(kMostScore, s) : s;
}

// Four codes (bytes of w; int8 ones with the sign bit flipped) to four fp16 values, exactly.
template <bool kE4m3>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kE4m3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {   // 1024 + (code + 128) has the code's bits as its last eight; then less 1152
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(w, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(w, 0x64646464u, 0x4342)), "r"(0x64806480u));
  }
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float scale) {
  return pack_f16x2(bf16_lo(w) * scale, bf16_hi(w) * scale);
}

// The map of a K or V cache, rows of dh (bf16: halves of 64), 128-byte swizzle (64-byte for
// 64-byte rows): boxes of `keys` rows of `heads` KV heads, one head after the other.
inline bool tree_cache_map(const TreeArgs& a, const void* cache, int dh, bool codes, int keys, int heads,
                           CUtensorMap* map) {
  const uint64_t es = codes ? 1 : 2, rows = static_cast<uint64_t>(a.batch) * a.cap;
  const uint64_t dims[3] = {static_cast<uint64_t>(dh), rows, static_cast<uint64_t>(a.n_hkv)};
  const uint64_t str[2] = {static_cast<uint64_t>(a.n_hkv) * dh * es, dh * es};
  const uint32_t box[3] = {static_cast<uint32_t>(codes ? dh : 64), static_cast<uint32_t>(keys),
                           static_cast<uint32_t>(heads)};
  return encode_tmap(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, cache, dims,
                     str, box, codes && dh == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// tree_rows.cu: the part over a cache of codes for up to kTreeRowsMax rows.
constexpr int kTreeRowsMax = 16;
int tree_rows_ctas(int rows);    // CTAs that fill the machine
int tree_rows_warps(int rows);   // warps of a CTA: hw * kw is at most these
tg_status launch_tree_rows(const TreeArgs& a, int head_dim, tg_dtype cache_dtype, cudaStream_t stream);

}  // namespace tg

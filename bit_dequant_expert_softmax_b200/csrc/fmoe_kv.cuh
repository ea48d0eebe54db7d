// The paged 4-bit key/value cache for sm_100a: filling it (rotation and quantisation on
// the way) and reading it back.
//
// Layout: include/fmoe_attn.h.  A tile is 16 tokens of one key/value head; a token's code
// row has its words in the order [8-channel block j][64-channel group g], so that a thread
// holding block j of every group reads one contiguous piece: with the mma.sync fragments of
// the attention kernel, thread t of a quad takes the 2 D/64 words of blocks 2t, 2t+1 of a key
// row, and thread g of eight the D/64 words of block g of a value row.
//
// Both kernels move bytes and nothing else bounds them: every row is read once in 16-byte
// (append) or 4-byte (gather) pieces per lane, contiguous over the lanes of a head row, and
// written once.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fmoe_attn.h"
#include "fmoe_device.cuh"

namespace fmoe {

constexpr int kKvTile = 16;      // tokens of a cache tile
constexpr int kKvThreads = 256;

template <int D>
struct KvGeom {
  static_assert(D == 64 || D == 128, "head sizes the cache is laid out for");
  static constexpr int kGroups = D / 64;                 // (scale, bias) words per row
  static constexpr int kRow = D / 2;                     // code bytes of a token
  static constexpr int kOffV = kKvTile * kRow;           // value codes
  static constexpr int kOffKs = 2 * kOffV;               // key (scale, bias) words
  static constexpr int kOffVs = kOffKs + kKvTile * kGroups * 4;
  static constexpr int kTileBytes = kOffVs + kKvTile * kGroups * 4;
  static constexpr int kLanes = D / 8;                   // lanes of a head row, 8 channels each
};

__host__ __device__ inline int64_t kv_page_bytes(int kv_heads, int D, int page_tokens) {
  return static_cast<int64_t>(kv_heads) * (page_tokens / kKvTile) * (kKvTile * (D + D / 8));
}

__device__ __forceinline__ void kv_error(uint32_t* err, uint32_t bit) {
  if (err != nullptr) atomicOr(err, bit);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

struct KvAppendParams {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const float* rope;
  const int32_t* positions;
  const int64_t* slots;
  uint8_t* cache;
  long long pages, page_bytes;
  uint16_t *q_out, *k_out;
  uint32_t* err;
  int rope_positions, rotary, q_heads, kv_heads, page_tokens;
};

// One token per block (blockIdx.x), its heads (queries, keys, values in this order) over
// the block's lane groups and blockIdx.y.  A lane owns 8 channels of a head row, which is
// one code word; a group's minimum and maximum are reduced over its 8 lanes.  The token's
// cosines and sines of the lane's channels are loaded once for all of its heads.
template <int D>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  using Gm = KvGeom<D>;
  constexpr int kPer = kKvThreads / Gm::kLanes;  // head rows in flight per block
  grid_launch_dependents();
  grid_dependency_wait();
  const long long tok = blockIdx.x;
  const long long slot = __ldg(p.slots + tok);
  if (slot < 0) return;
  const long long page = slot / p.page_tokens;
  if (page >= p.pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0) kv_error(p.err, FMOE_DEVERR_BAD_SLOT);
    return;
  }
  const int place = static_cast<int>(slot - page * p.page_tokens);
  const int lane = threadIdx.x % Gm::kLanes, grp = threadIdx.x / Gm::kLanes;
  const int half = p.rotary / 2, c0 = lane * 8;
  const bool turned = c0 < p.rotary, first = c0 < half;
  float cs[8], sn[8];
  if (p.rotary > 0) {
    const int pos = __ldg(p.positions + tok);
    if (pos < 0 || pos >= p.rope_positions) {
      if (threadIdx.x == 0 && blockIdx.y == 0) kv_error(p.err, FMOE_DEVERR_BAD_POSITION);
      return;
    }
    if (turned) {
      const float4* row = reinterpret_cast<const float4*>(p.rope + static_cast<long long>(pos) * p.rotary +
                                                          (first ? c0 : c0 - half));
      const float4 a = __ldg(row), b = __ldg(row + 1);
      const float4 c = __ldg(row + half / 4), d = __ldg(row + half / 4 + 1);
      cs[0] = a.x, cs[1] = a.y, cs[2] = a.z, cs[3] = a.w, cs[4] = b.x, cs[5] = b.y, cs[6] = b.z, cs[7] = b.w;
      sn[0] = c.x, sn[1] = c.y, sn[2] = c.z, sn[3] = c.w, sn[4] = d.x, sn[5] = d.y, sn[6] = d.z, sn[7] = d.w;
    }
  }
  uint8_t* tile0 = p.cache + page * p.page_bytes + static_cast<long long>(place / kKvTile) * Gm::kTileBytes;
  const long long head_bytes = static_cast<long long>(p.page_tokens / kKvTile) * Gm::kTileBytes;
  const int row = place % kKvTile, grp64 = lane / 8;
  const int h_q = p.q != nullptr ? 0 : p.q_heads;
  const int heads = p.q_heads + 2 * p.kv_heads;
  for (int h0 = h_q + blockIdx.y * kPer; h0 < heads; h0 += kPer * gridDim.y) {  // uniform over the block
    const int h = h0 + grp;
    const bool live = h < heads;
    const int kind = h < p.q_heads ? 0 : h < p.q_heads + p.kv_heads ? 1 : 2;
    const int hk = kind == 0 ? h : kind == 1 ? h - p.q_heads : h - p.q_heads - p.kv_heads;
    const uint16_t* src = (kind == 0 ? p.q + tok * p.q_stride : kind == 1 ? p.k + tok * p.k_stride : p.v + tok * p.v_stride) +
                          static_cast<long long>(hk) * D;
    const bool turn = live && turned && kind < 2;
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
    if (live) x = *reinterpret_cast<const uint4*>(src + c0);
    if (turn) y = *reinterpret_cast<const uint4*>(src + (first ? c0 + half : c0 - half));
    __syncwarp();  // a row rotated in place is read by all of its lanes before any writes
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (turn) {
      const uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // products and sum rounded one by one (no contraction): the result does not
        // depend on which half of the pair a lane holds
        const float p0 = __fmul_rn(bf16_lo(z[i]), sn[2 * i]), p1 = __fmul_rn(bf16_hi(z[i]), sn[2 * i + 1]);
        const float a0 = __fmul_rn(bf16_lo(w[i]), cs[2 * i]), a1 = __fmul_rn(bf16_hi(w[i]), cs[2 * i + 1]);
        w[i] = first ? pack_bf16(__fsub_rn(a0, p0), __fsub_rn(a1, p1)) : pack_bf16(__fadd_rn(a0, p0), __fadd_rn(a1, p1));
      }
    }
    uint16_t* dst = kind == 0 ? p.q_out : kind == 1 ? p.k_out : nullptr;
    if (live && dst != nullptr)
      *reinterpret_cast<uint4*>(dst + (tok * (kind == 0 ? p.q_heads : p.kv_heads) + hk) * D + c0) =
          make_uint4(w[0], w[1], w[2], w[3]);
    // the group's quantisation (query rows go through it too where a warp holds both)
    if (__any_sync(0xffffffffu, live && kind > 0)) {
      float lo = bf16_lo(w[0]), hi = lo;
      uint32_t odd = 0;  // an infinity or a NaN
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo = fminf(lo, fminf(bf16_lo(w[i]), bf16_hi(w[i])));
        hi = fmaxf(hi, fmaxf(bf16_lo(w[i]), bf16_hi(w[i])));
        odd |= (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
      }
#pragma unroll
      for (int off = 1; off < 8; off *= 2) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        odd |= __shfl_xor_sync(0xffffffffu, odd, off);
      }
      // halves: max - min of finite bf16 may pass the largest float, their halves' cannot
      const float lo2 = 0.5f * lo;
      const float s = bf16_lo(pack_bf16(__fdiv_rn(__fsub_rn(0.5f * hi, lo2), 7.5f), 0.f));
      const float s2 = 0.5f * s;
      uint32_t code = 0;
      if (odd == 0 && s > 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float r0 = rintf(__fdiv_rn(__fsub_rn(0.5f * bf16_lo(w[i]), lo2), s2));
          const float r1 = rintf(__fdiv_rn(__fsub_rn(0.5f * bf16_hi(w[i]), lo2), s2));
          code |= static_cast<uint32_t>(fminf(r0, 15.f)) << (8 * i);
          code |= static_cast<uint32_t>(fminf(r1, 15.f)) << (8 * i + 4);
        }
      }
      if (live && kind > 0) {
        uint8_t* tile = tile0 + hk * head_bytes;
        uint8_t* crow = tile + (kind == 2 ? Gm::kOffV : 0) + row * Gm::kRow;
        reinterpret_cast<uint32_t*>(crow)[(lane & 7) * Gm::kGroups + grp64] = code;
        if ((lane & 7) == 0) {
          const uint32_t sb = odd ? 0x7FC00000u : (__float_as_uint(s) >> 16) | (__float_as_uint(lo) & 0xFFFF0000u);
          reinterpret_cast<uint32_t*>(tile + (kind == 2 ? Gm::kOffVs : Gm::kOffKs))[row * Gm::kGroups + grp64] = sb;
        }
      }
    }
  }
}

struct KvGatherParams {
  const uint8_t* cache;
  long long pages, page_bytes, rows;
  const int32_t *table, *first, *cu;
  uint16_t *k_out, *v_out;
  uint32_t* err;
  int width, seqs, kv_heads, page_tokens;
};

constexpr int kKvGatherRows = 16;  // rows per block

// kKvGatherRows packed rows per block (blockIdx.x), heads over blockIdx.y.  The first
// threads find each row's place in the cache (-1: none); then a lane group takes one head's
// keys or values of one row.
template <int D>
__global__ void __launch_bounds__(kKvThreads) kv_gather_kernel(const __grid_constant__ KvGatherParams p) {
  using Gm = KvGeom<D>;
  constexpr int kPer = kKvThreads / Gm::kLanes;
  __shared__ long long where[kKvGatherRows];
  __shared__ int first_seq;
  grid_launch_dependents();
  grid_dependency_wait();
  const long long r0 = static_cast<long long>(blockIdx.x) * kKvGatherRows;
  // the sequence of row r0: the number of sequences that end at or before it
  int ended = 0;
  for (int i = threadIdx.x; i < p.seqs; i += kKvThreads) ended += __ldg(p.cu + i + 1) <= r0;
  if (threadIdx.x == 0) first_seq = 0;
  __syncthreads();
  ended = __reduce_add_sync(0xffffffffu, ended);
  if ((threadIdx.x & 31) == 0 && ended) atomicAdd(&first_seq, ended);
  __syncthreads();
  if (threadIdx.x < kKvGatherRows) {
    const long long r = r0 + threadIdx.x;
    long long at = -1;
    if (r < p.rows) {
      int s = first_seq;
      while (s < p.seqs && __ldg(p.cu + s + 1) <= r) ++s;
      if (s < p.seqs) {
        const int lo = __ldg(p.cu + s), t0 = p.first != nullptr ? __ldg(p.first + s) : 0;
        const long long t = t0 + (r - lo);
        if (r < lo || t0 < 0 || t / p.page_tokens >= p.width) {
          kv_error(p.err, FMOE_DEVERR_BAD_LENGTH);
        } else {
          const int page = __ldg(p.table + static_cast<long long>(s) * p.width + t / p.page_tokens);
          if (page < 0 || page >= p.pages) {
            kv_error(p.err, FMOE_DEVERR_BAD_PAGE);
          } else {
            const int place = static_cast<int>(t % p.page_tokens);
            at = page * p.page_bytes + static_cast<long long>(place / kKvTile) * Gm::kTileBytes + place % kKvTile;
          }
        }
      }
    }
    where[threadIdx.x] = at;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && __ldg(p.cu + p.seqs) > p.rows)
    kv_error(p.err, FMOE_DEVERR_BAD_LENGTH);
  __syncthreads();
  const int lane = threadIdx.x % Gm::kLanes, grp = threadIdx.x / Gm::kLanes;
  const long long head_bytes = static_cast<long long>(p.page_tokens / kKvTile) * Gm::kTileBytes;
  for (int h = blockIdx.y; h < p.kv_heads; h += gridDim.y) {
#pragma unroll
    for (int i = grp; i < 2 * kKvGatherRows; i += kPer) {
      const int rr = i >> 1;
      const bool val = i & 1;
      const long long at = where[rr];
      if (at < 0) continue;
      // page and tile offsets are multiples of 16, the row in the tile rides in the low bits
      const int row = static_cast<int>(at & 15);
      const uint8_t* tile = p.cache + (at - row) + h * head_bytes;
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(tile + (val ? Gm::kOffV : 0) + row * Gm::kRow) + (lane & 7) * Gm::kGroups + lane / 8);
      const uint32_t sb = __ldg(reinterpret_cast<const uint32_t*>(tile + (val ? Gm::kOffVs : Gm::kOffKs)) + row * Gm::kGroups + lane / 8);
      const float s = sb_scale(sb), b = sb_bias(sb);
      uint32_t o[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        o[c] = pack_bf16(fmaf(s, static_cast<float>((w >> (8 * c)) & 15u), b), fmaf(s, static_cast<float>((w >> (8 * c + 4)) & 15u), b));
      uint16_t* dst = (val ? p.v_out : p.k_out) + ((r0 + rr) * p.kv_heads + h) * D + lane * 8;
      *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace fmoe

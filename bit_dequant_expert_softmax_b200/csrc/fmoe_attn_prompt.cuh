// Causal attention over packed prompts (sm_100a): o_i = softmax_j(scale q_i . k_j) v_j over the
// keys j <= i + Lk - Lq of the query's own sequence, one pass over the keys per block of
// query rows with the running maximum and sum of each row in registers.
#pragma once

#include "fmoe_attn_decode.cuh"

namespace fmoe {

constexpr int kApRows = 128;
constexpr int kApKeys = 64;
constexpr int kApThreads = 256;

struct ApParams {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride, q_rows, k_rows;
  const int32_t *cu_q, *cu_k;
  uint16_t* out;
  uint32_t* err;
  float scale_log2;
  int seqs, q_heads, kv_heads, group, tile_tokens;
};

// The sequence and first query of row block `tile` of the packed sequences' line of blocks;
// false behind the last one.  Every warp finds it for itself.
struct ApTile {
  int q0, nq, k0, nk;  // the sequence's rows
  int first;           // the block's first query in it
};
__device__ __forceinline__ bool ap_span(const int32_t* cu, int s, long long rows, int& lo, int& n) {
  lo = __ldg(cu + s);
  const int hi = __ldg(cu + s + 1);
  n = hi - lo;
  if (lo < 0 || hi < lo || hi > rows) {
    n = 0;
    return false;
  }
  return true;
}
__device__ __forceinline__ bool ap_find(const ApParams& p, long long tile, ApTile& r) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  for (int s0 = 0; s0 < p.seqs; s0 += 32) {
    int q0 = 0, nq = 0, k0 = 0, nk = 0;
    if (s0 + lane < p.seqs) {
      const bool a = ap_span(p.cu_q, s0 + lane, p.q_rows, q0, nq), b = ap_span(p.cu_k, s0 + lane, p.k_rows, k0, nk);
      if (!a || !b) {
        nq = 0;
        kv_error(p.err, FMOE_DEVERR_BAD_LENGTH);
      }
    }
    const int mine = (nq + p.tile_tokens - 1) / p.tile_tokens;
    long long upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + upto > tile);
    if (past != 0) {
      const int who = __ffs(past) - 1;
      r.q0 = __shfl_sync(0xffffffffu, q0, who);
      r.nq = __shfl_sync(0xffffffffu, nq, who);
      r.k0 = __shfl_sync(0xffffffffu, k0, who);
      r.nk = __shfl_sync(0xffffffffu, nk, who);
      r.first = static_cast<int>(tile - (base + __shfl_sync(0xffffffffu, upto - mine, who))) * p.tile_tokens;
      return true;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// A block takes 128 rows of one key/value head, row = token * G + query head of the group
// (tile_tokens = 128 / G tokens), a warp 16 of them; the keys go by 64.
template <int D>
__global__ void __launch_bounds__(kApThreads) attn_prompt_kernel(const __grid_constant__ ApParams p) {
  constexpr int kPitch = D + 8;
  __shared__ __align__(16) uint16_t sk[kApKeys][kPitch], sv[kApKeys][kPitch];
  grid_launch_dependents();
  grid_dependency_wait();
  ApTile T;
  if (!ap_find(p, blockIdx.x, T)) return;
  const int kvh = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // rows g and g + 8 of the warp's 16
  int tok[2], head[2];
  bool live[2];
  int sees[2];
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = warp * 16 + g + 8 * h;
    tok[h] = T.first + row / p.group;
    head[h] = kvh * p.group + row % p.group;
    live[h] = row < p.tile_tokens * p.group && tok[h] < T.nq;
    sees[h] = live[h] ? tok[h] + T.nk - T.nq + 1 : 0;  // keys [0, sees)
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + (T.q0 + tok[h]) * p.q_stride + static_cast<long long>(head[h]) * D);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      qf[c][h] = live[h] ? __ldg(src + 8 * c + t) : 0u;
      qf[c][h + 2] = live[h] ? __ldg(src + 8 * c + t + 4) : 0u;
    }
  }
  const int last = min(T.nq, T.first + p.tile_tokens) - 1;
  const int keys = max(0, min(T.nk, last + T.nk - T.nq + 1));
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  for (int j0 = 0; j0 < keys; j0 += kApKeys) {
    __syncthreads();
    for (int i = threadIdx.x; i < kApKeys * (D / 8); i += kApThreads) {
      const int r = i / (D / 8), c = i % (D / 8) * 8;
      uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
      if (j0 + r < keys) {
        a = __ldg(reinterpret_cast<const uint4*>(p.k + (T.k0 + j0 + r) * p.k_stride + static_cast<long long>(kvh) * D + c));
        b = __ldg(reinterpret_cast<const uint4*>(p.v + (T.k0 + j0 + r) * p.v_stride + static_cast<long long>(kvh) * D + c));
      }
      *reinterpret_cast<uint4*>(&sk[r][c]) = a;
      *reinterpret_cast<uint4*>(&sv[r][c]) = b;
    }
    __syncthreads();
    float s[kApKeys / 8][4];
#pragma unroll
    for (int i = 0; i < kApKeys / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int i = 0; i < kApKeys / 16; ++i) {
        uint32_t b[4];
        ldmatrix4(b, smem_u32(&sk[16 * i + (lane & 7) + (lane >> 4) * 8][16 * c + ((lane >> 3) & 1) * 8]));
        mma_bf16(s[2 * i], qf[c][0], qf[c][1], qf[c][2], qf[c][3], b[0], b[1]);
        mma_bf16(s[2 * i + 1], qf[c][0], qf[c][1], qf[c][2], qf[c][3], b[2], b[3]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < kApKeys / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = s[i][2 * h + e];
          x = j0 + 8 * i + 2 * t + e < sees[h] ? x * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float now = fmaxf(m[h], mx), ref = now == -INFINITY ? 0.f : now, al = ex2(m[h] - ref);
      m[h] = now;
      l[h] *= al;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][2 * h] *= al;
        o[i][2 * h + 1] *= al;
      }
#pragma unroll
      for (int i = 0; i < kApKeys / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = s[i][2 * h + e];
          x = ex2(x - ref);
          l[h] += x;
        }
    }
#pragma unroll
    for (int c = 0; c < kApKeys / 16; ++c) {
      const uint32_t a0 = pack_bf16(s[2 * c][0], s[2 * c][1]), a1 = pack_bf16(s[2 * c][2], s[2 * c][3]);
      const uint32_t a2 = pack_bf16(s[2 * c + 1][0], s[2 * c + 1][1]), a3 = pack_bf16(s[2 * c + 1][2], s[2 * c + 1][3]);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t b[4];
        ldmatrix4_trans(b, smem_u32(&sv[16 * c + (lane & 15)][16 * i + (lane >> 4) * 8]));
        mma_bf16(o[2 * i], a0, a1, a2, a3, b[0], b[1]);
        mma_bf16(o[2 * i + 1], a0, a1, a2, a3, b[2], b[3]);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (!live[h]) continue;
    const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + ((T.q0 + tok[h]) * static_cast<long long>(p.q_heads) + head[h]) * D);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) dst[4 * i + t] = pack_bf16(o[i][2 * h] * inv, o[i][2 * h + 1] * inv);
  }
}

}  // namespace fmoe

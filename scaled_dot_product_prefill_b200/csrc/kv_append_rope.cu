// kv_append_rope.cu -- rotate new tokens' q and k by position and store k and v in the paged cache.
//
// What is computed, for row t of a packed batch, the i-th of the n new tokens
// of sequence b, at position p = seq_lens[b] - n + i of its cache: every pair
// c < R / 2 of a head of q or k,
//     a' = a cos[p, c] - b sin[p, c],   b' = b cos[p, c] + a sin[p, c],
// with the pair at columns (c, c + R / 2), or (2 c, 2 c + 1) when interleaved;
// columns from R on are kept.  The rotated q goes to q_out, the rotated k to
// slot p % page_size of page page_table[b][p / page_size] (and to k_out), v
// to the same slot unchanged.  cos and sin come from a table in fp32 that the
// caller forms (in whatever precision its angles need, with whatever scaling
// of the frequencies).  The products are formed in fp32, one of the two
// of each sum exactly (fma), and rounded once, to bf16 or to an E4M3 code.
//
// How.  The work is a copy with a few operations on the way, bound by HBM:
// each q, k, v element is read once and written once, 16 bytes at a time.  A
// warp takes one token and, per step, 32 / U of its head rows (q, then k, then
// v), U = D / 16 lanes to a row: a lane owns 16 columns, both halves of the
// pairs of 8 consecutive table columns, so that a rotation never leaves the
// lane and the lane's 8 cosines and 8 sines serve all its STEPS rows.  All rows'
// loads are issued before anything that depends on the position, whose
// chain (sequence, length, then page and angles) is the latency of a
// small call.  Blocks of 2 warps, 12 of them on an SM: 24 warps keep 96 KB of
// loads in flight, where the registers of a free choice left 16 warps (130 us
// on 30.6 k tokens, 768 MB, against 117 us, 6.5 TB/s, the measured copy rate; at 80
// registers the interleaved form spills 8 bytes), and
// blocks of 8 warps end less evenly (24.6 us on 5.4 k tokens, 134 MB, against 23.3).
#include <type_traits>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 64;

struct RopeParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_out;           // either may be null
  void *k_pool, *v_pool;
  const float* table;                     // [max_pos, R]: R/2 cosines, then R/2 sines
  const int32_t *cu, *page_table, *seq_lens;   // cu null: n_each tokens of every sequence
  unsigned int* err;
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int B, T, n_each, Hq, Hkv, D, R, page_size, num_pages, max_pages, max_pos;
  int groups;                             // warps per token
  long long row_warps;                    // T * groups
  float k_inv, v_inv;
};

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16* p) {
  // not the read-only path: q_out may be q, k_out may be k
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// 8 values -> 8 E4M3 codes of x * inv, nearest even, saturated at +-448 (as attn_kv_append_fp8).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned short pair;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(x[2 * i + 1] * inv), "f"(x[2 * i] * inv));
    out[i >> 1] |= static_cast<uint32_t>(pair) << (16 * (i & 1));
  }
  return make_uint2(out[0], out[1]);
}

// Number of sequences that end at or before row t (the index of the one that holds
// it, if any does): a 33-way search by the whole warp, one load per lane and level.
__device__ __forceinline__ int ends_before(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, n = B;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + (lane + 1) * step;
    const bool ended = (lane + 1) * step <= n && cu[i] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, ended));
    lo += c * step;
    n = min(step - 1, n - c * step);
  }
  return lo;
}

template <bool FP8, bool INTERLEAVED, int STEPS>
__global__ void __launch_bounds__(kThreads, STEPS > 1 ? 12 : 1) kv_append_rope_kernel(const RopeParams p) {
  grid_dependency_wait();   // the pools may still be read, and q, k, v written, by the kernel before
  grid_dependents_may_start();
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (w >= p.row_warps) {   // the warps behind those of the rows look the lengths over, 32 sequences each
    const long long b = (w - p.row_warps) * 32 + lane;
    if (p.cu != nullptr && b < p.B && (p.cu[b] < 0 || p.cu[b + 1] < p.cu[b] || p.cu[b + 1] > p.T))
      record_error(p.err, ATTN_ERRBIT_BADPAGE);
    return;
  }
  const int t = static_cast<int>(w / p.groups);
  const int group = static_cast<int>(w - static_cast<long long>(t) * p.groups);

  const int U = p.D / 16, per = 32 / U;            // lanes per row, rows per step
  const int u = lane % U, rows = p.Hq + 2 * p.Hkv;
  const bool turns = u < p.R / 16;
  // this lane's two runs of 8 columns
  const int c0 = (turns && !INTERLEAVED) ? 8 * u : 16 * u;
  const int c1 = (turns && !INTERLEAVED) ? p.R / 2 + 8 * u : 16 * u + 8;

  uint4 a[STEPS], b[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int row = (group * STEPS + s) * per + lane / U;
    if (lane >= per * U || row >= rows) continue;
    const __nv_bfloat16* src = row < p.Hq ? p.q + t * p.q_stride + static_cast<long long>(row) * p.D
                               : row < p.Hq + p.Hkv
                                   ? p.k + t * p.k_stride + static_cast<long long>(row - p.Hq) * p.D
                                   : p.v + t * p.v_stride + static_cast<long long>(row - p.Hq - p.Hkv) * p.D;
    a[s] = ld16(src + c0);
    b[s] = ld16(src + c1);
  }

  // the token's sequence and position; a row that no sequence holds stays as it is
  int seq, first, end;
  if (p.cu == nullptr) {
    seq = t / p.n_each;
    first = seq * p.n_each;
    end = first + p.n_each;
  } else {
    seq = ends_before(p.cu, p.B, t, lane);
    if (seq >= p.B) return;
    first = p.cu[seq];
    end = p.cu[seq + 1];
    // positions count from the sequence's end: one that is not wholly in the buffer has none to go by
    if (t < first || t >= end || first < 0 || end > p.T) {
      if (t >= p.cu[0] && lane == 0) record_error(p.err, ATTN_ERRBIT_BADPAGE);
      return;
    }
  }
  const long long at = static_cast<long long>(p.seq_lens[seq]) - end + t;
  if (at < 0) return;                       // the cache is shorter than the chunk: no position
  if (at >= p.max_pos) {
    if (lane == 0) record_error(p.err, ATTN_ERRBIT_BADPAGE);
    return;
  }
  const int pos = static_cast<int>(at);
  const int page = pos / p.page_size;
  const int phys = page < p.max_pages ? p.page_table[static_cast<size_t>(seq) * p.max_pages + page] : -1;
  float cs[8], sn[8];
  if (turns) {
    const float* row = p.table + static_cast<size_t>(pos) * p.R + 8 * u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 x = *reinterpret_cast<const float4*>(row + 4 * h);
      const float4 y = *reinterpret_cast<const float4*>(row + p.R / 2 + 4 * h);
      cs[4 * h] = x.x, cs[4 * h + 1] = x.y, cs[4 * h + 2] = x.z, cs[4 * h + 3] = x.w;
      sn[4 * h] = y.x, sn[4 * h + 1] = y.y, sn[4 * h + 2] = y.z, sn[4 * h + 3] = y.w;
    }
  }
  const bool held = phys >= 0 && phys < p.num_pages;
  if (!held && lane == 0) record_error(p.err, ATTN_ERRBIT_BADPAGE);
  // element offset of (this slot, head 0) in the pools
  const size_t slot = (static_cast<size_t>(held ? phys : 0) * p.Hkv * p.page_size + (pos - page * p.page_size)) * p.D;

#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int row = (group * STEPS + s) * per + lane / U;
    if (lane >= per * U || row >= rows) continue;
    const bool is_v = row >= p.Hq + p.Hkv;
    if (turns && !is_v) {
      float x[8], y[8];
      unpack8(a[s], x);
      unpack8(b[s], y);
      float x2[8], y2[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (INTERLEAVED) {   // columns 2 e and 2 e + 1 of the lane's 16
          float& l = e < 4 ? x[2 * e] : y[2 * e - 8];
          float& h = e < 4 ? x[2 * e + 1] : y[2 * e - 7];
          const float rl = fmaf(l, cs[e], -(h * sn[e])), rh = fmaf(h, cs[e], l * sn[e]);
          (e < 4 ? x2[2 * e] : y2[2 * e - 8]) = rl;
          (e < 4 ? x2[2 * e + 1] : y2[2 * e - 7]) = rh;
        } else {
          x2[e] = fmaf(x[e], cs[e], -(y[e] * sn[e]));
          y2[e] = fmaf(y[e], cs[e], x[e] * sn[e]);
        }
      }
      if (row < p.Hq) {
        if (p.q_out != nullptr) {
          __nv_bfloat16* dst = p.q_out + t * p.q_out_stride + static_cast<long long>(row) * p.D;
          *reinterpret_cast<uint4*>(dst + c0) = pack8(x2);
          *reinterpret_cast<uint4*>(dst + c1) = pack8(y2);
        }
        continue;
      }
      const int g = row - p.Hq;
      if (p.k_out != nullptr) {
        __nv_bfloat16* dst = p.k_out + t * p.k_out_stride + static_cast<long long>(g) * p.D;
        *reinterpret_cast<uint4*>(dst + c0) = pack8(x2);
        *reinterpret_cast<uint4*>(dst + c1) = pack8(y2);
      }
      if (!held) continue;
      const size_t dst = slot + static_cast<size_t>(g) * p.page_size * p.D;
      if constexpr (FP8) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.k_pool) + dst + c0) = codes8(x2, p.k_inv);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.k_pool) + dst + c1) = codes8(y2, p.k_inv);
      } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_pool) + dst + c0) = pack8(x2);
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_pool) + dst + c1) = pack8(y2);
      }
      continue;
    }
    // columns that do not turn, and v: moved bit for bit (or encoded)
    if (row < p.Hq) {
      if (p.q_out != nullptr) {
        __nv_bfloat16* dst = p.q_out + t * p.q_out_stride + static_cast<long long>(row) * p.D;
        *reinterpret_cast<uint4*>(dst + c0) = a[s];
        *reinterpret_cast<uint4*>(dst + c1) = b[s];
      }
      continue;
    }
    const int g = is_v ? row - p.Hq - p.Hkv : row - p.Hq;
    if (!is_v && p.k_out != nullptr) {
      __nv_bfloat16* dst = p.k_out + t * p.k_out_stride + static_cast<long long>(g) * p.D;
      *reinterpret_cast<uint4*>(dst + c0) = a[s];
      *reinterpret_cast<uint4*>(dst + c1) = b[s];
    }
    if (!held) continue;
    const size_t dst = slot + static_cast<size_t>(g) * p.page_size * p.D;
    void* pool = is_v ? p.v_pool : p.k_pool;
    if constexpr (FP8) {
      float x[8], y[8];
      unpack8(a[s], x);
      unpack8(b[s], y);
      const float inv = is_v ? p.v_inv : p.k_inv;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + dst + c0) = codes8(x, inv);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + dst + c1) = codes8(y, inv);
    } else {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pool) + dst + c0) = a[s];
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pool) + dst + c1) = b[s];
    }
  }
}

template <bool FP8, bool INTERLEAVED>
cudaError_t launch(RopeParams& p, cudaStream_t stream) {
  const int per = 32 / (p.D / 16);
  const int steps = (p.Hq + 2 * p.Hkv + per - 1) / per;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // With few warp steps (decode steps, short prompts) each gets a warp, for the shortest chain; with many a
  // warp takes 4, for its loads in flight and one position chain to them.  us with 1 and with 4 at 5, 21,
  // 42 and 166 steps per SM (32/8 heads, D = 128, one decode step and 256 to 2048 tokens): 2.4 / 2.8,
  // 3.5 / 3.0, 4.1 / 3.3, 13.3 / 7.6; at 9, 17 and 69 (12/12, D = 64): 2.4 / 2.8, 2.7 / 3.0, 6.0 / 5.7.
  const bool few = static_cast<long long>(p.T) * steps <= static_cast<long long>(sms) * 16;
  const int take = few ? 1 : 4;
  p.groups = (steps + take - 1) / take;
  p.row_warps = static_cast<long long>(p.T) * p.groups;
  // (looking the lengths over in the rows' own warps slowed those: 127 us on 30.6 k tokens, against 120)
  const long long warps = p.row_warps + (p.cu != nullptr ? (p.B + 31LL) / 32 : 0);
  const long long blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  auto kern = few ? kv_append_rope_kernel<FP8, INTERLEAVED, 1> : kv_append_rope_kernel<FP8, INTERLEAVED, 4>;
  return launch_dependent(kern, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_kv_append_rope(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* k_pool,
                                  void* v_pool, const float* table, const int32_t* cu_seqlens,
                                  const int32_t* page_table, const int32_t* seq_lens, int page_size, int B, int T,
                                  int Hq, int Hkv, int D, int R, int interleaved, long long q_stride,
                                  long long k_stride, long long v_stride, long long q_out_stride,
                                  long long k_out_stride, int num_pages, int max_pages, int max_pos, unsigned int* err,
                                  cudaStream_t stream, bool fp8, float k_scale, float v_scale) {
  RopeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.table = table;
  p.cu = cu_seqlens;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.err = err;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.B = B;
  p.T = T;
  p.n_each = cu_seqlens == nullptr ? T / B : 0;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.R = R;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.max_pos = max_pos;
  p.k_inv = 1.f / k_scale;
  p.v_inv = 1.f / v_scale;
  if (fp8) return interleaved ? launch<true, true>(p, stream) : launch<true, false>(p, stream);
  return interleaved ? launch<false, true>(p, stream) : launch<false, false>(p, stream);
}

}  // namespace attn

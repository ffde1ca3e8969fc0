// Linear attention with a decay for each head, in chunks on the matrix cores.
//
// For one (sequence, head), S_0 given and a log decay g_t per step,
//   S_t = e^{g_t} S_{t-1} + v_s k_t v_t^T        (S: KD x VD)
//   o_t = o_s S_t^T q_t
// With G_i the sum of g over a chunk's steps up to i, the steps of a chunk of 32 are
//   o_i = o_s [ e^{G_i} S_0^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_s v_j ]
//   S'  = e^{G_31} S_0 + sum_j k_j (e^{G_31 - G_j} v_s v_j)^T.
// Every exponent is a difference over steps between j and i, never the quotient of two powers.
// A log decay of kReset or less is a decay of exactly zero in float32: it drops what came before
// by the index comparison j >= (last reset up to i), so a reset's size never enters G.
//
// The same recurrence, with its operands exchanged, gives the gradients (g the gradient of o,
// L_t that of S_t):  dq = LA(g, v, k) forward in time on S^T;  dk = LA(v, g, q) and
// dv = LA(k, q, g) backward in time on L^T and L, where a step's decay is that of the step after
// it and the state entering is the gradient of the final state. A launch runs one or more such
// roles (LinRole).
//
// Layout. One workgroup walks the chunks of one (role, sequence, head, segment of the time axis);
// wave w owns columns 32 w .. 32 w + 31 of the values, and its part of the state (KD x 32) stays
// in float32 accumulators of v_mfma_f32_32x32 for the whole walk: lane l holds column l % 32,
// accumulator r row 8 (r / 4) + 4 (l / 32) + r % 4 of each block of 32 rows. Products contract
// over an index in any order, so everything is contracted in that order: accumulators r = 8 s ..
// 8 s + 7 are, converted in place, the operand slice s of the next product (state and scores never
// pass through LDS), and the other operand is read from LDS as two runs of 4, at 16 s + 4 (l / 32)
// and 8 further. The scores are formed transposed (rows j, columns i), so that they too are
// operands where they stand; every wave forms them for itself, which costs 2 KD / 32 of its matrix
// instructions and saves a barrier and a trip through LDS. Operands with the step index along the
// registers (k^T, v^T) are read by the transposing LDS load (bf16) or element by element (float32).
//
// Tiles of q, k and v are copied global to LDS directly, a stage ahead, one barrier a chunk. LDS
// rows hold a power of two of bytes; their 16-byte chunks are permuted by row (lin_swizzle) so that
// the 16 rows (or 4 rows by 32 bytes) that the LDS serves together lie on distinct banks. Steps
// past the end and columns past the width are fetched from outside the buffer's extent: zeros.
//
// Precision. bf16 operands are exact; products accumulate in float32 and the state is float32.
// What has to be rounded to feed a bf16 product (scores, the scaled values, the state as an
// operand) is split into NP, NV and NS bf16 terms, 8 bits of the mantissa each. float32 operands
// use the float32 matrix instructions, with no rounding.
//
// Causality holds for what is not finite too: a v_j that is infinite or NaN would reach the
// chunk's earlier rows as 0 * v_j, so a chunk with one adds its scores row by row.
#pragma once
#include "common.h"
#include "kernels.h"

namespace slstm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// log decays up to this are a decay of zero: e^-104 is below float32's smallest subnormal
constexpr float kReset = -104.0f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr uint32_t kLinOutside = 0x80000000u;  // a byte offset beyond every buffer extent
constexpr uint32_t kLinExtent = 0x7fffffffu;

typedef __attribute__((address_space(3))) void* lin_lds_t;

__device__ __forceinline__ rsrc_t lin_rsrc(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                           static_cast<int>(kLinExtent), 0x00020000);
}

// the permutation of a row's 16-byte chunks for rows of RB bytes
template <int RB>
__device__ __forceinline__ uint32_t lin_swizzle(uint32_t row) {
  constexpr int kShift = RB >= 256 ? 0 : RB == 128 ? 1 : 2;
  constexpr uint32_t kMask = RB >= 256 ? 7 : RB == 128 ? 3 : 1;
  return (((row >> kShift) & kMask) << 1) | ((row >> 3) & 1u);
}

__device__ __forceinline__ void lin_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // this wave's LDS accesses; global loads stay in flight
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void lin_wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// ---- operand slices: 8 values a lane, in the accumulators' row order --------------------------
template <bool BF16>
struct LinOps;

template <>
struct LinOps<true> {
  typedef bf16x8 frag;
  static constexpr int kSize = 2;

  static __device__ __forceinline__ f32x16 mma(const frag& a, const frag& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  // slice s of row `row` of a tile: elements 16 s + 4 half .. + 3 and 16 s + 8 + 4 half .. + 3
  template <int RB>
  static __device__ __forceinline__ frag row_slice(const unsigned char* tile, uint32_t row, uint32_t half, int s) {
    const uint32_t base = row * RB + (lin_swizzle<RB>(row) << 4) + 8 * half;
    union { u32x2 u[2]; frag f; } r;
    r.u[0] = *reinterpret_cast<const u32x2*>(tile + (base ^ static_cast<uint32_t>(s << 5)));
    r.u[1] = *reinterpret_cast<const u32x2*>(tile + (base ^ static_cast<uint32_t>((s << 5) | 16)));
    return r.f;
  }
  // slice s of column col0 + lane % 32: rows 16 s + 4 half .. + 3 and 16 s + 8 + 4 half .. + 3.
  // The transposing load gives lane i of 16 the column i of a 4 x 16 block whose rows lanes
  // 4 r .. 4 r + 3 address, 8 bytes each.
  template <int RB>
  static __device__ __forceinline__ frag column_slice(const unsigned char* tile, uint32_t col0, uint32_t lane, int s) {
    const uint32_t i = lane & 15u, half = lane >> 5;
    const uint32_t col = col0 + 16u * ((lane >> 4) & 1u) + 4u * (i & 3u);
    union { s16x4 v[2]; frag f; } r;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t row = 16u * s + 8u * e + 4u * half + (i >> 2);
      const uint32_t at = row * RB + (((col >> 3) ^ lin_swizzle<RB>(row)) << 4) + 2u * (col & 7u);
      r.v[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(const_cast<unsigned char*>(tile) + at));
    }
    return r.f;
  }
  static __device__ __forceinline__ float element(const unsigned char* tile, int RB, uint32_t swizzle, uint32_t row,
                                                  uint32_t col) {
    return bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + row * RB + (((col >> 3) ^ swizzle) << 4) + 2u * (col & 7u)));
  }
  static __device__ __forceinline__ f32x8 widen(const frag& f) {
    union { frag f; uint32_t u[4]; } r{f};
    f32x8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.u[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.u[i] & 0xffff0000u);
    }
    return v;
  }
  // v as N bf16 terms, each the rounding of what the ones before it leave
  template <int N>
  static __device__ __forceinline__ void split(f32x8 v, frag (&out)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      out[n] = __builtin_convertvector(v, frag);
      if (n + 1 < N) v -= widen(out[n]);
    }
  }
  // whether a slice holds an infinity or NaN
  static __device__ __forceinline__ bool not_finite(const frag& f) {
    union { frag f; uint32_t u[4]; } r{f};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      bad |= (r.u[i] & 0x7f800000u) == 0x7f800000u || (r.u[i] & 0x7f80u) == 0x7f80u;
    return bad;
  }
  // 4 values of a row of global memory at a byte offset, and back
  static __device__ __forceinline__ f32x4 load4(rsrc_t r, uint32_t off) {
    const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xffff0000u)};
  }
  typedef u32x2 packed4;
  static __device__ __forceinline__ packed4 pack4(float a, float b, float c, float d) {
    return u32x2{pack_bf16(a, b), pack_bf16(c, d)};
  }
  static __device__ __forceinline__ void store4(packed4 v, rsrc_t r, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b64(v, r, off, 0, 0);
  }
};

template <>
struct LinOps<false> {
  typedef f32x8 frag;
  static constexpr int kSize = 4;

  static __device__ __forceinline__ f32x16 mma(const frag& a, const frag& b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  template <int RB>
  static __device__ __forceinline__ frag row_slice(const unsigned char* tile, uint32_t row, uint32_t half, int s) {
    const uint32_t base = row * RB, sw = lin_swizzle<RB>(row);
    union { f32x4 v[2]; frag f; } r;
    r.v[0] = *reinterpret_cast<const f32x4*>(tile + base + (((4u * s + half) ^ sw) << 4));
    r.v[1] = *reinterpret_cast<const f32x4*>(tile + base + (((4u * s + 2u + half) ^ sw) << 4));
    return r.f;
  }
  template <int RB>
  static __device__ __forceinline__ frag column_slice(const unsigned char* tile, uint32_t col0, uint32_t lane, int s) {
    const uint32_t half = lane >> 5, col = col0 + (lane & 31u);
    frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t row = 16u * s + 8u * (e >> 2) + 4u * half + (e & 3);
      f[e] = *reinterpret_cast<const float*>(tile + row * RB + (((col >> 2) ^ lin_swizzle<RB>(row)) << 4) + 4u * (col & 3u));
    }
    return f;
  }
  static __device__ __forceinline__ float element(const unsigned char* tile, int RB, uint32_t swizzle, uint32_t row,
                                                  uint32_t col) {
    return *reinterpret_cast<const float*>(tile + row * RB + (((col >> 2) ^ swizzle) << 4) + 4u * (col & 3u));
  }
  static __device__ __forceinline__ f32x8 widen(const frag& f) { return f; }
  template <int N>
  static __device__ __forceinline__ void split(f32x8 v, frag (&out)[N]) {
    static_assert(N == 1, "float32 operands are not split");
    out[0] = v;
  }
  static __device__ __forceinline__ bool not_finite(const frag& f) {
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) bad |= (__float_as_uint(f[e]) & 0x7f800000u) == 0x7f800000u;
    return bad;
  }
  static __device__ __forceinline__ f32x4 load4(rsrc_t r, uint32_t off) {
    union { u32x4 u; f32x4 f; } v{__builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0)};
    return v.f;
  }
  typedef f32x4 packed4;
  static __device__ __forceinline__ packed4 pack4(float a, float b, float c, float d) { return f32x4{a, b, c, d}; }
  static __device__ __forceinline__ void store4(packed4 v, rsrc_t r, uint32_t off) {
    union { f32x4 f; u32x4 u; } t{v};
    __builtin_amdgcn_raw_buffer_store_b128(t.u, r, off, 0, 0);
  }
};

// ---- what a workgroup works on -----------------------------------------------------------------
struct LinItem {
  int seq, head, seg;
  int start;  // first step of the sequence in its row
  int len;    // its steps
  i64 row;    // batch row
  int slot;   // (sequence, segment) counted over all sequences
};

// Slots: unpacked, sequence b has n_seg of them; packed, sequence s has those from start / L + s
// on (never more than it needs: ceil(len / L) <= floor(end / L) - floor(start / L) + 1).
__device__ __forceinline__ bool lin_item(const LinLaunch& a, int slot, int head, LinItem& it) {
  it.head = head;
  it.slot = slot;
  if (a.cu == nullptr) {
    it.seq = slot / a.n_seg;
    it.seg = slot - it.seq * a.n_seg;
    it.start = 0;
    it.len = a.T;
    it.row = it.seq;
    return true;
  }
  auto first = [&](int s) { return min(max(a.cu[s], 0), a.T); };
  int lo = 0, hi = a.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first(mid) / a.seg_len + mid <= slot) lo = mid;
    else hi = mid - 1;
  }
  it.seq = lo;
  it.start = first(lo);
  it.len = max(0, min(max(a.cu[lo + 1], 0), a.T) - it.start);
  it.seg = slot - (it.start / a.seg_len + lo);
  it.row = 0;
  return it.seg >= 0 && (it.seg == 0 || it.seg < (it.len + a.seg_len - 1) / a.seg_len);
}

// ---- the walk ------------------------------------------------------------------------------------
// KB, VB: blocks of 32 columns of keys and values (powers of two: LDS rows). kFull: outputs and
// final states; otherwise only each segment's own contribution to the state and its decay.
template <bool BF16, int KB, int VB, bool kFull, int NS, int NP, int NV>
__global__ __launch_bounds__(64 * VB, 2) void linear_walk_kernel(const LinLaunch a) {
  typedef LinOps<BF16> Ops;
  typedef typename Ops::frag frag;
  constexpr int kSize = Ops::kSize;
  constexpr int RBK = KB * 32 * kSize, RBV = VB * 32 * kSize;
  constexpr int kTileK = 32 * RBK, kTileV = 32 * RBV;
  constexpr int kStage = (kFull ? 2 : 1) * kTileK + kTileV;
  // two stages where LDS holds them (as two objects: the compiler then sees which one is being filled)
  constexpr bool kTwo = 2 * kStage <= 144 * 1024;
  __shared__ __attribute__((aligned(1024))) unsigned char st0[kStage];
  __shared__ __attribute__((aligned(1024))) unsigned char st1[kTwo ? kStage : 16];
  __shared__ __attribute__((aligned(16))) float gates[VB][2][32];  // G_j and the weights w_j, a copy a wave
  __shared__ float dots[2][VB][32];

  const int lane = threadIdx.x & 63;
  const int wave = VB == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t half = static_cast<uint32_t>(lane) >> 5, li = static_cast<uint32_t>(lane) & 31u;

  // workgroup -> (role, head, slot): the roles of an item follow each other on the same XCD
  const int bid = blockIdx.x;
  const int n_items = a.n_slots * a.H;
  int role, item;
  if (a.n_roles == 1) {
    role = 0;
    item = bid;
  } else {
    const int xcd = bid & 7, idx = bid >> 3;
    role = idx % a.n_roles;
    item = (idx / a.n_roles) * 8 + xcd;
  }
  if (item >= n_items) return;
  LinItem it;
  if (!lin_item(a, item / a.H, item % a.H, it)) return;
  const LinRole& R = a.role[role];
  const int KD = R.KD, VD = R.VD;
  const int p_begin = it.seg * a.seg_len;
  const int p_end = min(it.len, p_begin + a.seg_len);
  const int n_chunks = max(0, (p_end - p_begin + 31) >> 5);
  if (!kFull && p_end >= it.len) return;  // nothing follows a sequence's last segment

  const i64 item_q = it.row * R.q.sb + it.start * R.q.st + it.head * R.q.sh;
  const i64 item_k = it.row * R.k.sb + it.start * R.k.st + it.head * R.k.sh;
  const i64 item_v = it.row * R.v.sb + it.start * R.v.st + it.head * R.v.sh;

  // lowest step of the chunk at position p0, and the step of its row r relative to that
  auto low_step = [&](int p0) { return R.reverse ? max(it.len - 32 - p0, 0) : p0; };
  auto row_step = [&](int p0, int r) { return R.reverse ? it.len - 1 - p0 - r - max(it.len - 32 - p0, 0) : r; };

  // one tile: 1 KiB blocks (1024 / RB rows) dealt to the waves; lane l fills slot l % (RB / 16) of
  // its block's row, that is, fetches the chunk which the permutation puts there
  auto issue_tile = [&](const LinView& v, i64 item_off, int width, int p0, unsigned char* dst, auto rb) {
    constexpr int RB = decltype(rb)::value;
    constexpr int kChunks = RB / 16;
    constexpr int kBlocks = 32 * RB / 1024;
    const rsrc_t r = lin_rsrc(static_cast<const char*>(v.data) + (item_off + static_cast<i64>(low_step(p0)) * v.st) * kSize);
#pragma unroll
    for (int i = 0; i < (kBlocks + VB - 1) / VB; ++i) {
      const int blk = i * VB + wave;
      if (kBlocks % VB != 0 && blk >= kBlocks) break;
      const uint32_t row = static_cast<uint32_t>(blk * (1024 / RB)) + static_cast<uint32_t>(lane) / kChunks;
      const uint32_t c = (static_cast<uint32_t>(lane) % kChunks) ^ lin_swizzle<RB>(row);
      const int col = static_cast<int>(c) * (16 / kSize);
      const bool in = p0 + static_cast<int>(row) < p_end && col < width;
      const uint32_t off = in ? static_cast<uint32_t>(row_step(p0, static_cast<int>(row))) * static_cast<uint32_t>(v.st * kSize) + col * kSize
                              : kLinOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lin_lds_t)(dst + blk * 1024), 16, off, 0, 0, 0);
    }
  };
  auto issue = [&](unsigned char* stg, int p0) {
    issue_tile(R.k, item_k, KD, p0, stg, std::integral_constant<int, RBK>{});
    issue_tile(R.v, item_v, VD, p0, stg + kTileK, std::integral_constant<int, RBV>{});
    if constexpr (kFull) issue_tile(R.q, item_q, KD, p0, stg + kTileK + kTileV, std::integral_constant<int, RBK>{});
  };
  // log decay entering position p (in base 2), 0 past the end; backward in time the step after it
  const float* gate = a.gate + it.row * a.gate_b + it.start * a.gate_t + it.head * a.gate_h;
  auto load_gate = [&](int p) -> float {
    if (p >= p_end || (R.reverse && p == 0)) return 0.0f;
    const int step = R.reverse ? it.len - p : p;
    return gate[step * a.gate_t];
  };

  // ---- the state this segment starts from ----
  const int col = wave * 32 + static_cast<int>(li);
  f32x16 S[KB];
  const float* from = nullptr;
  i64 rs = VD, cs = 1;
  if (kFull && it.seg > 0) {
    from = R.seg_states + (static_cast<i64>(it.slot - 1) * a.H + it.head) * KD * VD;
  } else if (kFull && R.state_in != nullptr) {
    from = R.state_in + (static_cast<i64>(it.seq) * a.H + it.head) * KD * VD;
    if (R.transposed) rs = 1, cs = KD;
  }
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int k = kb * 32 + 8 * (r >> 2) + 4 * static_cast<int>(half) + (r & 3);
      S[kb][r] = (from != nullptr && k < KD && col < VD) ? from[k * rs + col * cs] : 0.0f;
    }
  float seg_decay = 1.0f;

  typename Ops::packed4 held[4];  // the chunk's outputs, stored after the next barrier
  const i64 item_o = kFull ? it.row * R.out.sb + it.start * R.out.st + it.head * R.out.sh : 0;
  auto store_held = [&](int p0) {
    const rsrc_t r = lin_rsrc(static_cast<const char*>(R.out.data) + (item_o + static_cast<i64>(low_step(p0)) * R.out.st) * kSize);
    const bool in = p0 + static_cast<int>(li) < p_end;
    const uint32_t row_off = static_cast<uint32_t>(row_step(p0, static_cast<int>(li))) * static_cast<uint32_t>(R.out.st * kSize);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = wave * 32 + 8 * i + 4 * static_cast<int>(half);
      Ops::store4(held[i], r, in && c < VD ? row_off + c * kSize : kLinOutside);
    }
    // the inner products of the outputs with R.dot's rows, the waves' parts in order
    if (R.dot_out != nullptr && wave == 0 && lane < 32 && in) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < VB; ++w) s += dots[(p0 >> 5) & 1][w][lane];
      const int step = low_step(p0) + row_step(p0, lane);
      R.dot_out[(it.row * a.H + it.head) * static_cast<i64>(a.T) + it.start + step] = s;
    }
  };

  auto chunk = [&](unsigned char* stg, int p0, float g) {
    const unsigned char* tk = stg;
    const unsigned char* tv = stg + kTileK;
    const unsigned char* tq = stg + kTileK + kTileV;
    // ---- decays of the chunk: lanes li = i hold G_i; copies for the rows j through LDS ----
    const uint32_t resets = static_cast<uint32_t>(__ballot(g <= kReset));
    float G = g <= kReset ? 0.0f : g * kLog2e;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float up = __shfl_up(G, off, 32);
      if (li >= static_cast<uint32_t>(off)) G += up;
    }
    const uint32_t upto = resets & (0xffffffffu >> (31u - li));
    const int since = 31 - __clz(static_cast<int>(upto));  // last reset up to i, -1 without one
    const int since_end = 31 - __clz(static_cast<int>(resets));
    const float G_end = __shfl(G, 31, 32);
    const float w = static_cast<int>(li) >= since_end ? __builtin_amdgcn_exp2f(G_end - G) * R.v_scale : 0.0f;
    const float decay = since_end >= 0 ? 0.0f : __builtin_amdgcn_exp2f(G_end);
    if (lane < 32) {
      gates[wave][0][lane] = G;
      gates[wave][1][lane] = w;
    }
    __builtin_amdgcn_wave_barrier();
    float wj[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 t = *reinterpret_cast<const f32x4*>(&gates[wave][1][8 * i + 4 * half]);
      wj[4 * i] = t.x, wj[4 * i + 1] = t.y, wj[4 * i + 2] = t.z, wj[4 * i + 3] = t.w;
    }
    frag vt[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) vt[s] = Ops::template column_slice<RBV>(tv, wave * 32, lane, s);

    if constexpr (kFull) {
      const float e_i = since >= 0 ? 0.0f : __builtin_amdgcn_exp2f(G);
      f32x16 P, O;
#pragma unroll
      for (int r = 0; r < 16; ++r) P[r] = 0.0f, O[r] = 0.0f;
      // scores k_j . q_i and what the state adds, S^T q_i
#pragma unroll
      for (int s = 0; s < 2 * KB; ++s) {
        const frag q = Ops::template row_slice<RBK>(tq, li, half, s);
        const frag k = Ops::template row_slice<RBK>(tk, li, half, s);
        P = Ops::mma(k, q, P);
        f32x8 sv;
#pragma unroll
        for (int e = 0; e < 8; ++e) sv[e] = S[s >> 1][8 * (s & 1) + e];
        frag sf[NS];
        Ops::template split<NS>(sv, sf);
#pragma unroll
        for (int n = NS - 1; n >= 0; --n) O = Ops::mma(sf[n], q, O);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 t = *reinterpret_cast<const f32x4*>(&gates[wave][0][8 * i + 4 * half]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * i + 4 * static_cast<int>(half) + e;
          const bool in = j <= static_cast<int>(li) && j >= since;
          const float d = __builtin_amdgcn_exp2f(G - t[e]) * R.v_scale;
          P[4 * i + e] = in ? P[4 * i + e] * d : 0.0f;
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) O[r] *= e_i;
      if (__ballot(Ops::not_finite(vt[0]) || Ops::not_finite(vt[1])) == 0) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          f32x8 pv;
#pragma unroll
          for (int e = 0; e < 8; ++e) pv[e] = P[8 * s + e];
          frag pf[NP];
          Ops::template split<NP>(pv, pf);
#pragma unroll
          for (int n = NP - 1; n >= 0; --n) O = Ops::mma(vt[s], pf[n], O);
        }
      } else {
// row by row, the accumulators of P passing through its first one
#pragma unroll 1
        for (int r = 0; r < 16; ++r) {
          const float mine = P[0], other = __shfl_xor(P[0], 32, 64);
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            const int j = 8 * (r >> 2) + 4 * hh + (r & 3);
            const float p = static_cast<int>(half) == hh ? mine : other;
            if (j <= static_cast<int>(li) && j >= since) {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                O[c] = fmaf(p, Ops::element(tv, RBV, lin_swizzle<RBV>(j), j, wave * 32 + 8 * (c >> 2) + 4 * half + (c & 3)), O[c]);
            }
          }
#pragma unroll
          for (int e = 0; e + 1 < 16; ++e) P[e] = P[e + 1];
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) O[r] *= R.o_scale;
      if (R.dot_out != nullptr) {
        const rsrc_t r = lin_rsrc(static_cast<const char*>(R.dot.data) +
                                  (it.row * R.dot.sb + it.start * R.dot.st + it.head * R.dot.sh + static_cast<i64>(low_step(p0)) * R.dot.st) * kSize);
        const bool in = p0 + static_cast<int>(li) < p_end;
        const uint32_t row_off = static_cast<uint32_t>(row_step(p0, static_cast<int>(li))) * static_cast<uint32_t>(R.dot.st * kSize);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = wave * 32 + 8 * i + 4 * static_cast<int>(half);
          const f32x4 t = Ops::load4(r, in && c < VD ? row_off + c * kSize : kLinOutside);
#pragma unroll
          for (int e = 0; e < 4; ++e) s = fmaf(t[e], O[4 * i + e], s);
        }
        s += __shfl_xor(s, 32, 64);
        if (lane < 32) dots[(p0 >> 5) & 1][wave][lane] = s;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) held[i] = Ops::pack4(O[4 * i], O[4 * i + 1], O[4 * i + 2], O[4 * i + 3]);
    }

    // ---- the state after the chunk ----
    frag vw[2][NV];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x8 v = Ops::widen(vt[s]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= wj[8 * s + e];
      Ops::template split<NV>(v, vw[s]);
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
      for (int r = 0; r < 16; ++r) S[kb][r] *= decay;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const frag kt = Ops::template column_slice<RBK>(tk, kb * 32, lane, s);
#pragma unroll
        for (int n = NV - 1; n >= 0; --n) S[kb] = Ops::mma(kt, vw[s][n], S[kb]);
      }
    }
    seg_decay *= decay;
  };

  // ---- the walk: the loads of chunk c + 1 are in flight while chunk c is computed ----
  float g_next = load_gate(p_begin + static_cast<int>(li));
  auto step = [&](int c, unsigned char* cur, unsigned char* refill) {
    const int p0 = p_begin + 32 * c;
    const float g = g_next;
    lin_wait_loads();
    lin_barrier();
    if (kFull && c > 0) store_held(p0 - 32);
    if (c + 1 < n_chunks) {
      g_next = load_gate(p0 + 32 + static_cast<int>(li));
      if constexpr (kTwo) issue(refill, p0 + 32);
    }
    chunk(cur, p0, g);
    if constexpr (!kTwo) {
      lin_barrier();
      if (c + 1 < n_chunks) issue(cur, p0 + 32);
    }
  };
  if (n_chunks > 0) issue(st0, p_begin);
  if constexpr (kTwo) {
    int c = 0;
    for (; c + 2 <= n_chunks; c += 2) {
      step(c, st0, st1);
      step(c + 1, st1, st0);
    }
    if (c < n_chunks) step(c, st0, st1);
  } else {
    for (int c = 0; c < n_chunks; ++c) step(c, st0, st0);
  }
  if (kFull && n_chunks > 0) {
    lin_barrier();  // the waves' inner products of the last chunk
    store_held(p_begin + 32 * (n_chunks - 1));
  }

  // ---- the state the segment ends with ----
  if constexpr (!kFull) {
    float* to = R.seg_states + (static_cast<i64>(it.slot) * a.H + it.head) * KD * VD;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int k = kb * 32 + 8 * (r >> 2) + 4 * static_cast<int>(half) + (r & 3);
        if (k < KD && col < VD) to[k * VD + col] = S[kb][r];
      }
    if (threadIdx.x == 0) R.seg_decays[static_cast<i64>(it.slot) * a.H + it.head] = seg_decay;
  } else if (p_end >= it.len) {
    // the gradient of the initial state also passes the first step's decay
    float lead = 1.0f;
    if (R.reverse && it.len > 0) lead = gate[0] <= kReset ? 0.0f : __builtin_amdgcn_exp2f(gate[0] * kLog2e);
    const i64 at = (static_cast<i64>(it.seq) * a.H + it.head) * KD * VD;
    if (R.state_out != nullptr) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int k = kb * 32 + 8 * (r >> 2) + 4 * static_cast<int>(half) + (r & 3);
          if (k < KD && col < VD) R.state_out[at + k * VD + col] = S[kb][r] * lead;
        }
    }
    if (R.edge_out != nullptr) {  // <edge, S>, the edge stored transposed
      float s = 0.0f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int k = kb * 32 + 8 * (r >> 2) + 4 * static_cast<int>(half) + (r & 3);
          if (k < KD && col < VD) s = fmaf(R.edge[at + static_cast<i64>(col) * KD + k], S[kb][r], s);
        }
      s = wave_sum(s);
      lin_barrier();
      if (lane == 0) dots[0][wave][0] = s;
      lin_barrier();
      if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < VB; ++w) s += dots[0][w][0];
        R.edge_out[static_cast<i64>(it.seq) * a.H + it.head] = s;
      }
    }
  }
}

// ---- launches ------------------------------------------------------------------------------------
template <bool BF16, int KB, int VB>
hipError_t lin_launch(const LinLaunch& a, LinPass pass, hipStream_t st) {
  const long long items = static_cast<long long>(a.n_slots) * a.H;
  const long long blocks = a.n_roles == 1 ? items : (items + 7) / 8 * 8 * a.n_roles;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * VB);
  constexpr int NF = BF16 ? 2 : 1;  // the forward: bf16 outputs, so one term for scores and state
  constexpr int NB = BF16 ? 3 : 1;  // the float32 gradient of the decay: float32 precision throughout
  switch (pass) {
    case LinPass::kStates: linear_walk_kernel<BF16, KB, VB, false, 1, 1, NB><<<grid, block, 0, st>>>(a); break;
    case LinPass::kForward: linear_walk_kernel<BF16, KB, VB, true, 1, 1, NF><<<grid, block, 0, st>>>(a); break;
    case LinPass::kExact: linear_walk_kernel<BF16, KB, VB, true, NB, NB, NB><<<grid, block, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

template <int KB>
hipError_t lin_launch_keys(bool bf16, int vb, const LinLaunch& a, LinPass pass, hipStream_t st) {
  switch (vb) {
    case 1: return bf16 ? lin_launch<true, KB, 1>(a, pass, st) : lin_launch<false, KB, 1>(a, pass, st);
    case 2: return bf16 ? lin_launch<true, KB, 2>(a, pass, st) : lin_launch<false, KB, 2>(a, pass, st);
    case 4: return bf16 ? lin_launch<true, KB, 4>(a, pass, st) : lin_launch<false, KB, 4>(a, pass, st);
    case 8: return bf16 ? lin_launch<true, KB, 8>(a, pass, st) : lin_launch<false, KB, 8>(a, pass, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace slstm

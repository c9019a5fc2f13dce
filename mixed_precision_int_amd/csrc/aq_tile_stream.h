// Streaming the packed tiles of one 16-row group: device code for kernels
// whose waves walk a tile row by themselves.
//
// Every tile is fetched by the same three buffer loads, whatever its
// precision: two 16-byte loads of codes and the row scales.  The buffer
// descriptor's size makes them conditional without a branch: an INT4 tile's
// second load, and every load of a column past the range, lie outside the
// descriptor, touch no memory and return zeros.  So the number of loads in
// flight is known at every point, the compiler waits for one stage of a
// pipeline at a time instead of for all loads, and a zero scale keeps a
// column that does not exist out of the sums.  (With branches around the
// loads it waited for every earlier load before each branch that reused a
// register: gate/up of 32 experts of 4096 x 1536, M = 32: 95 us.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "aq_device.h"
#include "aq_internal.h"

namespace aq {

__device__ __forceinline__ v4i load16(const void *p) { return *reinterpret_cast<const v4i *>(p); }

// A value at a wave-uniform address that this kernel does not write, through
// the scalar cache.
template <typename T>
__device__ __forceinline__ T uload(const T *p) {
  return *(const __attribute__((address_space(4))) T *)(uintptr_t)p;
}

// A packed projection as kernel arguments.
struct Packed {
  const uint32_t *labels;
  const int32_t *off4, *off8;
  const uint8_t *w4, *w8;
  const float *s4, *s8;
  int C, T4, T8, label_words;
};
inline Packed packed_of(const PackedView &v) {
  Packed p;
  p.labels = reinterpret_cast<const uint32_t *>(v.labels);
  p.off4 = v.off4; p.off8 = v.off8;
  p.w4 = v.w4; p.w8 = reinterpret_cast<const uint8_t *>(v.w8);
  p.s4 = v.s4; p.s8 = v.s8;
  p.C = v.C; p.T4 = v.T4; p.T8 = v.T8;
  p.label_words = (int)(((long long)v.R * v.C + 31) / 32);
  return p;
}

// One lane's share of a 16-row group of a tile.  INT4: a holds both nibbles
// and b is zero.
struct Tile {
  v4i a, b;
  float sc;
  int is4;
};

constexpr int kNT = 2;  // buffer-load cache policy: non-temporal

// Labels of tiles t .. t + 63 of a projection (those past its last word are
// not of the row that asks).
struct LabelWords {
  uint32_t l0, l1, l2;
  int sh;
  __device__ __forceinline__ LabelWords(const Packed &p, int t) {
    const int w0 = t >> 5, last = p.label_words - 1;
    l0 = uload(p.labels + min(w0, last));
    l1 = uload(p.labels + min(w0 + 1, last));
    l2 = uload(p.labels + min(w0 + 2, last));
    sh = t & 31;
  }
  __device__ __forceinline__ uint64_t bits() const {
    const uint64_t x = (uint64_t)l0 | ((uint64_t)l1 << 32);
    return sh ? (x >> sh) | ((uint64_t)l2 << (64 - sh)) : x;
  }
};

// What a walk of tile row r starts from: five scalar loads.  Several rows'
// are made before the first walk, so that they travel together.
struct RowMeta {
  int tb, o4, o8;
  LabelWords w;
  __device__ __forceinline__ RowMeta(const Packed &p, int r)
      : tb(r * p.C), o4(uload(p.off4 + r)), o8(uload(p.off8 + r)), w(p, r * p.C) {}
};

// The tiles of columns c0 .. c1-1 of a tile row, rows 16rg .. 16rg+15: lane l
// gets row l % 16, k-group l / 16.  Indices by eq. 16; an index outside the
// buffers (inconsistent metadata) reads as a zero tile.
template <int BK>
struct RowStream {
  const Packed &p;
  int tb, idx4, idx8, j, c1, wb;
  uint64_t win;  // labels of columns wb .. wb + 63
  int g, row16, row4;

  __device__ __forceinline__ uint64_t window(int t) const { return LabelWords(p, t).bits(); }

  __device__ __forceinline__ RowStream(const Packed &p_, const RowMeta &m, int rg, int c0, int c1_, int lane)
      : p(p_), tb(m.tb), j(c0), c1(c1_), wb(0), win(m.w.bits()), g(lane >> 4) {
    row16 = rg * 256 + (lane & 15) * 16;
    row4 = row16 >> 2;
    int n4 = 0, c = c0;
    while (c >= 64) {  // rows of more than 64 tile columns
      n4 += __popcll(win);
      wb += 64;
      c -= 64;
      win = window(tb + wb);
    }
    n4 += __popcll(win & ((1ull << c) - 1ull));
    idx4 = m.o4 + n4;
    idx8 = m.o8 + (c0 - n4);
  }

  __device__ __forceinline__ void fetch(Tile &t) {
    if (j < c1 && j - wb >= 64) {
      wb = j;
      win = window(tb + wb);
    }
    const int is4 = (int)(win >> ((j - wb) & 63)) & 1;
    const int idx = is4 ? idx4 : idx8;
    const bool live = j < c1 && (unsigned)idx < (unsigned)(is4 ? p.T4 : p.T8);
    idx4 += is4;
    idx8 += is4 ^ 1;
    ++j;
    constexpr int B4 = 32 * BK, B8 = 64 * BK;
    const uint8_t *base = is4 ? p.w4 + (size_t)idx * B4 : p.w8 + (size_t)idx * B8;
    const float *sbase = (is4 ? p.s4 : p.s8) + (size_t)idx * 64;
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, live ? (is4 ? B4 : B8) : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(sbase), 0, live ? 256 : 0, 0x00020000);
    t.is4 = is4;
    if (BK == 128) {
      // INT8: panels 2g and 2g + 1; INT4: panel g, its second load out of range
      const int off = (g << (is4 ? 10 : 11)) + row16;
      t.a = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rw, off, 0, kNT));
      t.b = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rw, off + (is4 ? B4 : 1024), 0, kNT));
    } else {
      // INT8: panel g; INT4: 8 bytes of panel g / 2 (each load out of range
      // for the other precision)
      typedef int v2i __attribute__((ext_vector_type(2)));
      t.a = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rw, (g << 10) + row16 + (is4 ? B4 : 0), 0, kNT));
      const v2i n = __builtin_bit_cast(
          v2i, __builtin_amdgcn_raw_buffer_load_b64(rw, ((g >> 1) << 10) + 8 * (g & 1) + row16 + (is4 ? 0 : B8), 0, kNT));
      t.b = v4i{n[0], n[1], 0, 0};
    }
    t.sc = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, row4, 0, 0));
  }
};

// The lane's share of 16 token rows for one tile column; x points at the
// lane's token row, column j * BK.  At b_K = 64 the columns an INT4 tile takes
// differ from an INT8 tile's.
template <int BK>
struct TileX {
  v4i a, b;
  __device__ __forceinline__ void load(const int8_t *x, int g) {
    if (BK == 128) {
      a = load16(x + 32 * g);
      b = load16(x + 32 * g + 16);
    } else {
      const int8_t *c = x + 32 * (g >> 1) + 8 * (g & 1);
      const uint2 p0 = *reinterpret_cast<const uint2 *>(c), p1 = *reinterpret_cast<const uint2 *>(c + 16);
      a = load16(x + 16 * g);
      b = v4i{(int)p0.x, (int)p0.y, (int)p1.x, (int)p1.y};
    }
  }
};

// The tile's MFMA operands.  INT4 codes are widened x16 (exact; scale_of takes
// it back): with is4 uniform, shift and masks are scalars and no lane selects.
template <int BK>
struct TileOp {
  v4i w0, w1;
  __device__ __forceinline__ explicit TileOp(const Tile &t) {
    const int m0 = t.is4 ? (int)0xF0F0F0F0 : -1, m1 = t.is4 ? (int)0xF0F0F0F0 : 0, sh = t.is4 ? 4 : 0;
    if (BK == 128) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w0[i] = (t.a[i] << sh) & m0;
        w1[i] = (t.a[i] & m1) | t.b[i];
      }
    } else {
      // INT4: t.a is zero and t.b holds 8 bytes; INT8: t.b is zero
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w0[i] = t.a[i] | ((t.b[i] << 4) & (int)0xF0F0F0F0);
        w0[i + 2] = t.a[i + 2] | (t.b[i] & (int)0xF0F0F0F0);
      }
      w1 = w0;
    }
  }
};

// INT32 product of the tile with 16 token rows: element e of a lane is token
// 4 (lane / 16) + e of weight row lane % 16.
template <int BK>
__device__ __forceinline__ v4i tile_product(const TileOp<BK> &w, const TileX<BK> &x, int is4) {
  v4i acc = {0, 0, 0, 0};
  if (BK == 128) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(x.a, w.w0, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(x.b, w.w1, acc, 0, 0, 0);
  } else {
    v4i xo;
#pragma unroll
    for (int i = 0; i < 4; ++i) xo[i] = is4 ? x.b[i] : x.a[i];
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(xo, w.w0, acc, 0, 0, 0);
  }
  return acc;
}

// The row scale with the 1/16 of the INT4 widening.
__device__ __forceinline__ float scale_of(const Tile &t) { return t.sc * (t.is4 ? 0.0625f : 1.0f); }

}  // namespace aq

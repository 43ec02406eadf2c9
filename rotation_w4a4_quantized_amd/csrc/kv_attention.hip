// kv_attention: causal attention of a step's queries over the paged 8-bit
// cache, one pass over the keys and values.
//
//   s_j = (scale log2 e) sK[page] (q . ck_j),  p_j = 2^(s_j - m),  l = sum p_j
//   o   = (sum_j p_j sV[page] cv_j) / l
//
// with the running maximum m. Both products run on fp16 matrix instructions
// with fp32 accumulation. The codes are exact in fp16. A query row is scaled by
// a power of two to a largest value in [2^14, 2^15), so a bf16 query is exact
// down to 2^-29 of it; an fp32 or transformed one is rounded by 2^-11. The second
// product's left factor is fp16(2^13 p_j sV / vref), vref the largest sV so far: at
// most 2^13, rounded by 2^-11 relative at most down to 2^-27 of the largest weight
// and by 2^-38 of it below; bf16, with 2^-8, would round about as much as the output
// itself. vref is a row's own, over the blocks that hold a key of the row: a later
// page's scale, however large, leaves the row's weights as they are. Maxima, sums
// and accumulators are fp32.
//
// Scores are computed transposed (keys are the matrix rows, queries the
// columns): a lane then owns one query, its maximum, sum and rescaling need no
// exchange beyond the 4 lanes of a column, and the weights come out in the very
// lanes and order in which the second product wants its right factor (the k
// order of a matrix product is free as long as both factors share it).
#include <algorithm>
#include <cmath>

#include "kv_common.hpp"
#include "launch.hpp"

namespace rw4 {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr float kWeightScale = 8192.0f;   // 2^13
constexpr float kLog2e = 1.44269504088896341f;

// Two codes as fp16: `w` holds codes + 128, sel picks the two bytes. The bytes
// land in the mantissa of 1024, and 1024 + (c + 128) - 1152 = c is exact.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  const v2h off = {static_cast<_Float16>(1152.0f), static_cast<_Float16>(1152.0f)};
  const v2h h = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, w, SEL));
  return __builtin_bit_cast(uint32_t, h - off);
}
constexpr uint32_t kLow = 0x04010400u, kHigh = 0x04030402u;   // bytes 0, 1 and 2, 3

// 8 codes (bytes of a, then of b, plus 128 each) in order
__device__ __forceinline__ v8h code8(uint32_t a, uint32_t b) {
  const v4u w = {code_pair<kLow>(a), code_pair<kHigh>(a), code_pair<kLow>(b), code_pair<kHigh>(b)};
  return __builtin_bit_cast(v8h, w);
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// a / b for scales 0 <= a <= b, b >= kLeastScale, within 2 ulp. The quarter keeps
// the reciprocal, which gives no subnormal numbers, above 2^-126 for every b.
constexpr float kLeastScale = 7.52316385e-37f;   // 2^-120
__device__ __forceinline__ float ratio(float a, float b) {
  return (a * 0.25f) * __builtin_amdgcn_rcpf(b * 0.25f);
}

// 8 columns of an output row
__device__ __forceinline__ void store_row8(const KvAttnArgs& p, int64_t t, int hq, int d,
                                           const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = f32_to_bf16(v[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
  *reinterpret_cast<uint4*>(p.out + t * p.ldo + static_cast<int64_t>(hq) * p.c.dh + d) =
      make_uint4(w[0], w[1], w[2], w[3]);
}

// The parts that the keys are split into, and where their results are: averages, not
// sums, which could pass fp32's range where the values do not.
struct Split {
  float* o;        // [rows Hq][S][dh]: average of the part's values
  float2* ml;      // [rows Hq][S]: maximum (base-2), sum
  int64_t chunk;   // keys of a part, at most: part s has [s chunk, (s + 1) chunk)
  int parts;
  int least_rows, most_rows;   // takes requests of more than the first, up to the second
  int tokens;      // rows of a request in o and ml; 0: those of the batch
  int least;       // split kernel: least keys of a part (a multiple of unit)
  static constexpr int unit = 128;
  // split kernel: the keys of a part of a request with `keys` of them, however
  // many the call's bound allows
  __device__ __forceinline__ int64_t part_keys(int64_t keys) const {
    const int each = static_cast<int>(hi64(keys, 0)) / parts + 1;
    return lo64(max((each + unit - 1) / unit * unit, least), chunk);
  }
  // the row of o and ml of a request's token, row t of the batch
  __device__ __forceinline__ int64_t row(int b, int tok, int64_t t) const {
    return tokens ? static_cast<int64_t>(b) * tokens + tok : t;
  }
};

struct Request {
  int t0, count, tokens;   // first row, new tokens, those computed
  int64_t first_pos;       // position of the first new token
};

__device__ __forceinline__ Request request(const KvAttnArgs& p, int b) {
  int t0, t1;
  request_rows(p.cu_new, b, p.T, t0, t1);
  const int64_t most = lo64(p.max_kv, p.max_pages << p.c.lg_page);
  return {t0, t1 - t0, static_cast<int>(lo64(t1 - t0, p.max_new)),
          lo64(p.kv_len[b], most) - (t1 - t0)};
}

// the page of a block of 16 keys and its scales; id < 0: keys count as masked
struct Block {
  int id;
  float sk, sv;
};
__device__ __forceinline__ Block block_of(const KvAttnArgs& p, int b, int h, int64_t key, bool live) {
  Block r{-1, 0.0f, 0.0f};
  if (live) {
    const int id = p.page_table[b * p.max_pages + (key >> p.c.lg_page)];
    if (id >= 0 && id < p.c.n_pages) {
      const int64_t at = static_cast<int64_t>(id) * p.c.H + h;
      r = {id, p.c.k_scale[at], p.c.v_scale[at]};
    }
  }
  return r;
}

// A query row's factors for the k steps of the first product, in the order in
// which a lane reads 16 codes of a key: lane group g (of 4) holds elements
// 64 j + 16 g + 0..15. Returns the row's factor of the scores in base 2.
template <int DH>
__device__ __forceinline__ float load_query(const KvAttnArgs& p, int64_t t, int hq, bool live, int g,
                                            v8h (&frag)[DH / 32]) {
  float v[DH / 4];
#pragma unroll
  for (int j = 0; j < DH / 64; ++j) {
    const int64_t at = t * p.ldq + static_cast<int64_t>(hq) * DH + 64 * j + 16 * g;
    if (!live) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[16 * j + i] = 0.0f;
    } else if (p.f32) {
      const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 w = x[i];
        v[16 * j + 4 * i] = w.x; v[16 * j + 4 * i + 1] = w.y;
        v[16 * j + 4 * i + 2] = w.z; v[16 * j + 4 * i + 3] = w.w;
      }
    } else {
      const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 w = x[i];
        float* o = v + 16 * j + 8 * i;
        o[0] = bf16lo(w.x); o[1] = bf16hi(w.x); o[2] = bf16lo(w.y); o[3] = bf16hi(w.y);
        o[4] = bf16lo(w.z); o[5] = bf16hi(w.z); o[6] = bf16lo(w.w); o[7] = bf16hi(w.w);
      }
    }
  }
  if (p.rotate) {   // strides 1..8 and 64.. inside the lane, 16 and 32 across the lane groups
#pragma unroll
    for (int s = 1; s < DH / 4; s *= 2)
#pragma unroll
      for (int i = 0; i < DH / 4; ++i)
        if ((i & s) == 0) {
          const float a = v[i], c = v[i + s];
          v[i] = a + c;
          v[i + s] = a - c;
        }
#pragma unroll
    for (int o = 16; o < 64; o *= 2) {
      const float sg = (threadIdx.x & o) ? -1.0f : 1.0f;
#pragma unroll
      for (int i = 0; i < DH / 4; ++i) v[i] = fmaf(sg, v[i], __shfl_xor(v[i], o, 64));
    }
  }
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < DH / 4; ++i) mx = fmaxf(mx, fabsf(v[i]));
  mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
  mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
  const int up = mx > 0.0f ? 14 - __builtin_amdgcn_frexp_expf(mx) + 1 : 0;   // mx 2^up in [2^14, 2^15)
#pragma unroll
  for (int s = 0; s < DH / 32; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      frag[s][i] = static_cast<_Float16>(__builtin_amdgcn_ldexpf(v[16 * (s / 2) + 8 * (s & 1) + i], up));
  const float norm = p.rotate ? head_norm<DH>() : 1.0f;
  return __builtin_amdgcn_ldexpf(p.scale * kLog2e * norm, -up);
}

// ---------------------------------------------------------------- few rows: the keys are split
// One tile of 32 keys in registers: keys as the left factor (lane: key lane %
// 16 of each block of 16, 16 codes per load), values as VB = DH / 16 columns of
// 8 keys per lane.
template <int DH>
struct Tile {
  static constexpr int VW = DH / 64;   // words of VB bytes
  uint4 k[2][DH / 64];
  uint32_t v[8][VW];
};

// Kernel for requests of at most 16 NC rows. A workgroup takes one part of a
// request's keys for one key head, its waves a contiguous share of the part
// each; a wave streams 32 keys and values at a time from HBM straight into the
// registers that feed the matrix instructions (no LDS: nothing is shared) while
// the next 32 are on their way. The waves' results are joined in LDS, the parts'
// by combine_kernel.
// Bound by HBM: 64 unequal requests of up to 16384 keys, 8 key heads of 128, 1174
// MB in 230 us by trace (5.1 TB/s; a large copy reaches 5.2); 8 of up to 2048 keys
// and 32 heads, 84 MB in 27 us, and one of 131072 keys, 269 MB in 60 us, with the
// join of the parts. Three waves to a
// SIMD (at most 168 registers) take 28.1 us for 8 requests of 2048 keys and 32 heads,
// two 29.3; four would spill (71 us). A workgroup of eight waves takes 25.3 us there,
// of four 27.0, but for the 64 requests 250 and of four 241, for the long one 61.2 and
// 59.7; of two 41 us for 8 requests of 4096 keys and 32 rows of 128, of four 29.5. The
// largest forms (48 rows of 128: 428 registers, 32 of 256: all 512, 29 of them spilled)
// run one wave to a SIMD.
template <int DH, int NC, int NW>
__global__ __launch_bounds__(64 * NW, (NC * DH <= 128) ? 3 : 1) void split_kernel(KvAttnArgs p, Split sp) {
  constexpr int VB = DH / 16, VW = DH / 64, KS = DH / 32, LD = DH + 4;
  extern __shared__ float lds[];
  float* acc_s = lds;                             // [NW][16 NC][LD]
  float* m_s = lds + NW * 16 * NC * LD;           // [NW][16 NC]
  float* l_s = m_s + NW * 16 * NC;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const int h = blockIdx.x, b = blockIdx.y, part = blockIdx.z;
  const int group = p.Hq / p.c.H, lg = p.c.lg_page;
  const Request rq = request(p, b);
  const int rows = rq.tokens * group;
  if (rows <= sp.least_rows || rows > sp.most_rows) return;
  const int64_t keys = rq.first_pos + rq.tokens;          // of the last row
  const int64_t chunk = sp.part_keys(keys), c0 = part * chunk, c1 = lo64(keys, c0 + chunk);
  if (c0 > 0 && c0 >= keys) return;

  // this wave's keys: [k0, k0 + 32 n_tiles), cut at c1
  const int64_t len = hi64(c1 - c0, 0);
  const int per = static_cast<int>((len + 32 * NW - 1) / (32 * NW));   // tiles of a wave
  const int64_t k0 = c0 + static_cast<int64_t>(w) * per * 32;
  const int n_tiles = static_cast<int>(lo64(hi64((c1 - k0 + 31) / 32, 0), per));
  const Block mine = block_of(p, b, h, k0 + 16 * lane, lane < 2 * n_tiles && k0 + 16 * lane < c1);

  const int64_t head_stride = static_cast<int64_t>(DH) << lg;
  auto load = [&](Tile<DH>& t, int i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int id = max(__builtin_amdgcn_readlane(mine.id, 2 * i + k), 0);
      const int in_page = static_cast<int>((k0 + 32 * i + 16 * k) & ((1 << lg) - 1)) * DH;
      const int64_t at = (static_cast<int64_t>(id) * p.c.H + h) * head_stride + in_page;
      const int8_t* kp = p.c.k_codes + at;
      const int8_t* vp = p.c.v_codes + at;
#pragma unroll
      for (int j = 0; j < DH / 64; ++j)
        t.k[k][j] = *reinterpret_cast<const uint4*>(kp + (n * DH + 64 * j + 16 * g));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int8_t* x = vp + ((4 * g + r) * DH + VB * n);
        if constexpr (VW == 1) {
          t.v[4 * k + r][0] = *reinterpret_cast<const uint32_t*>(x);
        } else if constexpr (VW == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(x);
          t.v[4 * k + r][0] = u.x; t.v[4 * k + r][1] = u.y;
        } else {
          const uint4 u = *reinterpret_cast<const uint4*>(x);
          t.v[4 * k + r][0] = u.x; t.v[4 * k + r][1] = u.y;
          t.v[4 * k + r][2] = u.z; t.v[4 * k + r][3] = u.w;
        }
      }
    }
  };
  Tile<DH> cur, next;
  if (n_tiles > 0) load(cur, 0);

  // the wave's queries: column n of tile c is row 16 c + n = (token, head of the group)
  v8h q[NC][KS];
  float coef[NC];
  int64_t pos[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int r = 16 * c + n, tok = r / group, hg = r - tok * group;
    const bool live = r < rows;
    coef[c] = load_query<DH>(p, rq.t0 + (live ? tok : 0), h * group + hg, live, g, q[c]);
    pos[c] = rq.first_pos + tok;
  }
  float m[NC], l[NC], vref[NC];   // vref: the largest sV among the row's keys so far, or kLeastScale
  v4f acc[NC][VB];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    m[c] = -INFINITY;
    l[c] = 0.0f;
    vref[c] = kLeastScale;
#pragma unroll
    for (int d = 0; d < VB; ++d) acc[c][d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }

  auto compute = [&](Tile<DH>& t, int i) {
    const int64_t key0 = k0 + 32 * i;
    v4f s[NC][2];
#pragma unroll
    for (int c = 0; c < NC; ++c) s[c][0] = s[c][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < DH / 64; ++j) {
        const uint4 u = t.k[k][j];
        const uint32_t bias = 0x80808080u;
        const v8h k_lo = code8(u.x ^ bias, u.y ^ bias), k_hi = code8(u.z ^ bias, u.w ^ bias);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          s[c][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_lo, q[c][2 * j], s[c][k], 0, 0, 0);
          s[c][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k_hi, q[c][2 * j + 1], s[c][k], 0, 0, 0);
        }
      }
    const int id0 = __builtin_amdgcn_readlane(mine.id, 2 * i), id1 = __builtin_amdgcn_readlane(mine.id, 2 * i + 1);
    const float sk0 = lane_value(mine.sk, 2 * i), sk1 = lane_value(mine.sk, 2 * i + 1);
    const float sv0 = lane_value(mine.sv, 2 * i), sv1 = lane_value(mine.sv, 2 * i + 1);
    // keys past a row's own position, and of pages that are not there
    const bool masked = id0 < 0 || id1 < 0 || key0 + 32 > rq.first_pos + 1;
    bool grown = false;
    float m_new[NC], v_new[NC], own0[NC], own1[NC];   // sV of the blocks with keys of the row
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      s[c][0] *= coef[c] * sk0;
      s[c][1] *= coef[c] * sk1;
      own0[c] = sv0;
      own1[c] = sv1;
      if (masked) {
        // keys 4 g + r (block 0) and 16 + 4 g + r (block 1) up to the row's own stay
        const int upto = static_cast<int>(lo64(pos[c] - key0, 64)), left = upto - 4 * g;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (r > left || id0 < 0) s[c][0][r] = -INFINITY;
          if (16 + r > left || id1 < 0) s[c][1][r] = -INFINITY;
        }
        if (upto < 0) own0[c] = 0.0f;
        if (upto < 16) own1[c] = 0.0f;
      }
      v_new[c] = fmaxf(vref[c], fmaxf(own0[c], own1[c]));
      float mx = fmaxf(fmaxf(fmaxf(s[c][0][0], s[c][0][1]), fmaxf(s[c][0][2], s[c][0][3])),
                       fmaxf(fmaxf(s[c][1][0], s[c][1][1]), fmaxf(s[c][1][2], s[c][1][3])));
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      m_new[c] = fmaxf(m[c], mx);
      grown |= m_new[c] > m[c] || v_new[c] > vref[c];
    }
    if (__any(grown)) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float a = 1.0f;
        if (m_new[c] > m[c]) a = __builtin_amdgcn_exp2f(m[c] - m_new[c]);
        l[c] *= a;
        m[c] = m_new[c];
        if (v_new[c] > vref[c]) {   // vref is set in here: set after it, 48 rows of 128 take 494 registers
          a *= ratio(vref[c], v_new[c]);
          vref[c] = v_new[c];
        }
#pragma unroll
        for (int d = 0; d < VB; ++d) acc[c][d] *= a;
      }
    }
    v8h pw[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float base = m[c] == -INFINITY ? 0.0f : m[c];
      const float w0 = kWeightScale * ratio(own0[c], vref[c]), w1 = kWeightScale * ratio(own1[c], vref[c]);
      v4f p0, p1;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        p0[r] = __builtin_amdgcn_exp2f(s[c][0][r] - base);
        p1[r] = __builtin_amdgcn_exp2f(s[c][1][r] - base);
      }
      l[c] += ((p0[0] + p0[1]) + (p0[2] + p0[3])) + ((p1[0] + p1[1]) + (p1[2] + p1[3]));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        pw[c][r] = static_cast<_Float16>(p0[r] * w0);
        pw[c][4 + r] = static_cast<_Float16>(p1[r] * w1);
      }
    }
#pragma unroll
    for (int x = 0; x < VW; ++x) {
      uint32_t lo[4], hi[4];   // pairs of keys, bytes interleaved: columns 0, 1 and 2, 3
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t a = t.v[2 * r][x] ^ 0x80808080u, c = t.v[2 * r + 1][x] ^ 0x80808080u;
        lo[r] = __builtin_amdgcn_perm(c, a, 0x05010400u);
        hi[r] = __builtin_amdgcn_perm(c, a, 0x07030602u);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v4u f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t y = e < 2 ? lo[r] : hi[r];
          f[r] = (e & 1) ? code_pair<kHigh>(y) : code_pair<kLow>(y);
        }
        const v8h vt = __builtin_bit_cast(v8h, f);
#pragma unroll
        for (int c = 0; c < NC; ++c)
          acc[c][4 * x + e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vt, pw[c], acc[c][4 * x + e], 0, 0, 0);
      }
    }
  };
  for (int i = 0; i < n_tiles; i += 2) {
    if (i + 1 < n_tiles) load(next, i + 1);
    compute(cur, i);
    if (i + 1 < n_tiles) {
      if (i + 2 < n_tiles) load(cur, i + 2);
      compute(next, i + 1);
    }
  }

  // join the waves
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    l[c] += __shfl_xor(l[c], 16, 64);
    l[c] += __shfl_xor(l[c], 32, 64);
    if (g == 0) {
      m_s[w * 16 * NC + 16 * c + n] = m[c];
      l_s[w * 16 * NC + 16 * c + n] = l[c];
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    // the wave's share of the sum of all; its accumulators times that are at most 127
    // before the values' scale
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int u = 0; u < NW; ++u) top = fmaxf(top, m_s[u * 16 * NC + 16 * c + n]);
#pragma unroll
    for (int u = 0; u < NW; ++u)
      sum += l_s[u * 16 * NC + 16 * c + n] * __builtin_amdgcn_exp2f(m_s[u * 16 * NC + 16 * c + n] - top);
    const float f = m[c] == -INFINITY ? 0.0f
                                      : __builtin_amdgcn_exp2f(m[c] - top) * __builtin_amdgcn_rcpf(sum * kWeightScale);
    const float unit_v = vref[c];
    // acc[c][d][i] is column VB (4 g + i) + d of row 16 c + n
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* o = acc_s + (w * 16 * NC + 16 * c + n) * LD + VB * (4 * g + i);
#pragma unroll
      for (int d = 0; d < VB; d += 4)
        *reinterpret_cast<float4*>(o + d) =
            make_float4(acc[c][d][i] * f * unit_v, acc[c][d + 1][i] * f * unit_v,
                        acc[c][d + 2][i] * f * unit_v, acc[c][d + 3][i] * f * unit_v);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < rows * (DH / 8); e += 64 * NW) {
    const int r = e / (DH / 8), d = (e - r * (DH / 8)) * 8, tok = r / group, hg = r - tok * group;
    const int64_t at_pos = rq.first_pos + tok;
    if (at_pos < c0 && part > 0) continue;        // the row has no key in this part
    float v[8] = {};
#pragma unroll
    for (int u = 0; u < NW; ++u) {
      const float* o = acc_s + (u * 16 * NC + r) * LD + d;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += o[i];
    }
    const int64_t t = rq.t0 + tok;
    const int hq = h * group + hg;
    if (at_pos < chunk) {                         // the row's keys are all in this part
      store_row8(p, t, hq, d, v);
    } else {
      const int64_t at = (sp.row(b, tok, t) * p.Hq + hq) * sp.parts + part;
      float4* o = reinterpret_cast<float4*>(sp.o + at * DH + d);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
      if (d == 0) {
        float top = -INFINITY, sum = 0.0f;
        for (int u = 0; u < NW; ++u) top = fmaxf(top, m_s[u * 16 * NC + r]);
        for (int u = 0; u < NW; ++u) {
          const float mu = m_s[u * 16 * NC + r];
          if (mu != -INFINITY) sum += l_s[u * 16 * NC + r] * __builtin_amdgcn_exp2f(mu - top);
        }
        sp.ml[at] = make_float2(top, sum);
      }
    }
  }
}

// ---------------------------------------------------------------- many rows: queries in tiles
// A query row's right factors of the 32 x 32 x 16 product: k step s holds
// elements 16 s + 8 g + 0..7 in the two lanes g = 0, 1 of a column. The loads are
// apart from the rest, so that they run while the pages are looked up.
template <int DH>
struct Query32 {
  uint4 raw[DH / 16][2];   // 8 values: bf16 in the first, or fp32 in both
};

template <int DH>
__device__ __forceinline__ void load_query32(const KvAttnArgs& p, int64_t t, int hq, bool live, int g,
                                             Query32<DH>& q) {
  const int64_t at = t * p.ldq + static_cast<int64_t>(hq) * DH + 8 * g;
#pragma unroll
  for (int s = 0; s < DH / 16; ++s) {
    q.raw[s][0] = q.raw[s][1] = make_uint4(0, 0, 0, 0);
    if (!live) continue;
    if (p.f32) {
      const uint4* x = reinterpret_cast<const uint4*>(static_cast<const float*>(p.q) + at + 16 * s);
      q.raw[s][0] = x[0];
      q.raw[s][1] = x[1];
    } else {
      q.raw[s][0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at + 16 * s);
    }
  }
}

// Returns the row's factor (>= 0) of the scores in base 2; the scale's sign is in
// the query.
template <int DH>
__device__ __forceinline__ float query_factors32(const KvAttnArgs& p, const Query32<DH>& q, int g,
                                                 v8h (&frag)[DH / 16]) {
  constexpr int N = DH / 16;
  float v[N][8];
#pragma unroll
  for (int s = 0; s < N; ++s) {
    const uint4 a = q.raw[s][0], b = q.raw[s][1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[s][i] = p.f32 ? __uint_as_float(w[i]) : (i & 1) ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
  }
  if (p.rotate) {   // strides 1, 2, 4 and 16.. inside the lane, 8 across the two lanes
    const float sg = g ? -1.0f : 1.0f;
#pragma unroll
    for (int s = 0; s < N; ++s) {
#pragma unroll
      for (int h = 1; h < 8; h *= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((i & h) == 0) {
            const float a = v[s][i], b = v[s][i + h];
            v[s][i] = a + b;
            v[s][i + h] = a - b;
          }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[s][i] = fmaf(sg, v[s][i], __shfl_xor(v[s][i], 32, 64));
    }
#pragma unroll
    for (int h = 1; h < N; h *= 2)
#pragma unroll
      for (int s = 0; s < N; ++s)
        if ((s & h) == 0)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = v[s][i], b = v[s + h][i];
            v[s][i] = a + b;
            v[s + h][i] = a - b;
          }
  }
  float mx = 0.0f;
#pragma unroll
  for (int s = 0; s < N; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[s][i]));
  mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
  const int up = mx > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(mx) : 0;
  const float sign = p.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
  for (int s = 0; s < N; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      frag[s][i] = static_cast<_Float16>(__builtin_amdgcn_ldexpf(v[s][i] * sign, up));
  const float norm = p.rotate ? head_norm<DH>() : 1.0f;
  return __builtin_amdgcn_ldexpf(fabsf(p.scale) * kLog2e * norm, -up);
}

// The phases of the tile kernel are inlined by declaration: in a function of its own a
// phase would reach LDS by flat accesses, for which a phase's barrier does not wait.
#define KV_INLINE __attribute__((always_inline))

// Keys and values of 64 keys in LDS as fp16, twice (one is filled while the
// other is read). Keys [64][DH], 16-byte pieces of a row at piece ^ (key % 16)
// (of 8 pieces for DH = 64: ^ key % 8). Values transposed, [DH][64], the 16
// keys of a product step in the order 0-3, 8-11 | 4-7, 12-15 in which the first
// product leaves the weights in the two lanes of a column, pieces at piece ^
// turn(d). Both orders keep the 16-byte reads of neighbouring lanes, and the
// 8-byte writes of the transposed values, on different banks.
__device__ __forceinline__ int turn(int d) { return (d ^ (d >> 3)) & 7; }

// the maximum that hands a NaN on: one instruction for three values, where fmaxf
// first quiets each input
__device__ __forceinline__ float maximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ float pair_max(float v) {   // with lane ^ 32
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return maximum(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

template <int N>
struct Int { static constexpr int value = N; };

// The order of N LDS reads that feed one matrix instruction each: kAhead reads
// stay ahead of the instruction that uses them.
constexpr int kAhead = 8;
template <int N>
__device__ __forceinline__ void reads_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
  for (int i = 0; i < N - kAhead; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
}

// Kernel for requests of more rows than the split kernel takes. A workgroup of
// NW waves takes 32 NW rows (tokens x heads of a group, so the heads of a group
// share what is staged) of one key head against one part of the keys; a wave
// takes 32 rows. The codes become fp16 once per workgroup on their way into LDS.
//
// A wave alternates between a matrix phase (the values' product of the last
// tile, the keys' product of this one) and a vector phase (softmax; staging).
// With 8 waves, two to a SIMD, the second four run one phase behind the first,
// so that one wave of each SIMD feeds the matrix cores while the other uses the
// vector unit; a barrier ends each phase. The first four stage the keys, the
// others the values, at the start of their matrix phases: with
// phase i (values of tile i, keys of tile i + 1) the first four write the keys of
// tile i + 2, whose buffer's keys of tile i the others have read a phase before,
// and the others a phase later the values of tile i + 1, which the first four
// read in the phase after.
//
// Bound by the two phases' alternation: a tile of 64 keys and 256 rows takes about
// 5300 cycles, of which a SIMD's matrix instructions need 2048 (counters: 38% busy), the
// LDS reads that feed them as many, and a wave's softmax 1500 to 1800; while a wave
// issues vector instructions, its SIMD's other wave gets few matrix instructions in
// (neither wave priorities nor swapped roles change that). 4096 new tokens, 32 heads of
// 128: 137.5 GFLOP in 173 us, 0.79 PFLOP/s of the 1.1 that a large fp16 library
// product reaches here; 2429 new tokens in three requests after up to 12000, 32 query
// and 8 key heads, in two parts: 309 GFLOP in 412 us, 0.75 PFLOP/s, 27 us of it the
// join.
//
// The maximum that the weights are relative to (mref) moves only when a new one
// exceeds it by 2^8: the accumulators are rescaled a few times in all. The
// scale of the values goes into the exponent, w = 2^(s - mref + log2(sV / vref)
// + 7), vref the largest sV of the row's keys so far (one for all rows of a wave
// until the tiles that some of them see in part), so a weight is at most 2^15 in
// fp16, exact to 2^-11 down to 2^-21 of the largest. A block's sum of w goes back to
// the sum of 2^(s - mref) by one factor. sV / vref counts as 2^-60 where it is less:
// such a weight is 0 in fp16.
template <int DH, int NW>
__global__ __launch_bounds__(64 * NW) void tile_kernel(KvAttnArgs p, Split sp, int items) {
  constexpr int KS = DH / 16, DB = DH / 32, PK = DH / 8;   // k steps, 32-column blocks, pieces of a key row
  constexpr bool TWO = NW == 8;                            // two groups of waves, a phase apart
  constexpr int SW = TWO ? NW / 2 : NW;                    // waves that stage keys, and values
  constexpr int PER = 64 * DH / 16 / (64 * SW);            // 16-code pieces of a thread
  extern __shared__ uint4 smem[];
  char* lds = reinterpret_cast<char*>(smem);               // keys [2][64][DH], values [2][DH][64]
  const int lane = threadIdx.x & 63, n = lane & 31, g = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = p.c.H, group = p.Hq / H, lg = p.c.lg_page;

  // Blocks are dealt to the 8 XCDs in turn: with a multiple of 8 heads, a head's
  // workgroups share one XCD's L2. The last tiles of a request, which see the
  // most keys, come first.
  const int L = blockIdx.x;
  const int h = (H & 7) == 0 ? (L & 7) + 8 * ((L >> 3) % (H >> 3)) : L % H;
  const int item = items - 1 - ((H & 7) == 0 ? (L >> 3) / (H >> 3) : L / H);
  const int part = blockIdx.y;
  constexpr int RT = 32 * NW;
  auto first_item = [&](int b) {
    return lo64(max(p.cu_new[b], 0), p.T) * group / RT + b;
  };
  const int b = wave_search(static_cast<int>(p.B), item, first_item);
  const Request rq = request(p, b);
  const int rows = rq.tokens * group;
  const int64_t first_row = (item - first_item(b)) * RT;
  if (rows <= sp.least_rows || first_row < 0 || first_row >= rows) return;
  const int R0 = static_cast<int>(first_row);
  const int last_tok = (min(R0 + RT, rows) - 1) / group;
  const int64_t keys = rq.first_pos + last_tok + 1;         // seen by the tile's last row
  const int64_t c0 = part * sp.chunk, c1 = lo64(keys, c0 + sp.chunk);
  if (c0 > 0 && c0 >= keys) return;
  const int n_tiles = static_cast<int>(hi64(c1 - c0 + 63, 0) / 64);

  const int r = R0 + 32 * w + n, tok = r / group, hg = r - tok * group;
  const bool live = r < rows;
  Query32<DH> query;
  load_query32<DH>(p, rq.t0 + (live ? tok : 0), h * group + hg, live, g, query);
  // positions from the part's first key on: the row's own, the least and the
  // most of the wave's rows (a wave past the rows has none)
  const int64_t pos = rq.first_pos + (live ? tok : last_tok);
  const int own_key = static_cast<int>(hi64(pos - c0, -1));
  const int least_key = static_cast<int>(hi64(rq.first_pos + min((R0 + 32 * w) / group, last_tok) - c0, -1));
  const int most_key = R0 + 32 * w < rows
      ? static_cast<int>(hi64(rq.first_pos + min((R0 + 32 * w + 31) / group, last_tok) - c0, -1)) : -1;
  const int active = min(n_tiles, (most_key + 64) / 64);    // tiles with keys for the wave's rows

  // pages and scales of 64 blocks of 16 keys (16 tiles), one per lane, and of
  // the next 64. at: the block's place in the cache in units of 16 keys (the
  // whole cache is below 2^31 of them), lv: log2 of sV, lt: the largest lv of the
  // four blocks of a tile; gone: bits of the blocks whose keys count as masked
  struct Blocks { int at; float sk, lv, lt; uint64_t gone; };
  auto blocks = [&](int window) {
    const int64_t key = c0 + 1024 * static_cast<int64_t>(window) + 16 * lane;
    const Block k = block_of(p, b, h, key, key < c1);
    const int64_t at = ((static_cast<int64_t>(max(k.id, 0)) * H + h) << (lg - 4)) +
                       ((key & ((1 << lg) - 1)) >> 4);
    const float lv = __builtin_amdgcn_logf(k.sv);
    float lt = fmaxf(lv, __shfl_xor(lv, 1, 64));
    lt = fmaxf(lt, __shfl_xor(lt, 2, 64));
    return Blocks{static_cast<int>(at), k.sk, lv, lt, __ballot(k.id < 0)};
  };
  Blocks cur = blocks(0), nxt = blocks(1);
  int window = 0;                                           // of cur
  v8h q[KS];
  const float coef = query_factors32<DH>(p, query, g, q);
  // byte offset in the codes of block blk of the tile that is loaded (its
  // window's places in k_at, v_at)
  int k_at = cur.at, v_at = cur.at;
  auto place = [&](int at, int blk) {
    return static_cast<int64_t>(__builtin_amdgcn_readlane(at, blk & 63)) * (16 * DH);
  };

  // Staging: 16 codes of a key's row; 8 columns of 4 neighbouring values (8 x 8
  // columns x 4 groups of keys x 2 blocks of 16 keys to a wave). The turned
  // pieces are byte offsets whose other pieces differ by an exclusive or.
  constexpr int VPER = DH >= 32 * SW ? DH / (32 * SW) : 1;  // pieces of values of a thread
  uint4 kraw[PER];
  uint2 vraw[VPER][4];
  const int ws = TWO ? w & (SW - 1) : w;
  constexpr int KR = 64 * 16 / DH;      // key rows of a wave's 64 pieces, in one block of 16
  constexpr int KBUF = 64 * DH * 2, VBASE = 2 * KBUF;
  constexpr int DW = DH / 64;           // waves along the columns
  const int w_key = ws * KR + lane / (DH / 16), w_d8 = (ws % DW) * 8 + (lane & 7), w_kk2 = ws / DW;
  const bool has_v = DH >= 32 * SW || w_kk2 < 2;            // for DH = 64 two waves suffice
  const int k_put = w_key * DH * 2 + 16 * ((2 * (lane % (DH / 16))) ^ (w_key & (PK >= 16 ? 15 : 7)));
  const int v_put = VBASE + w_d8 * 1024 + 8 * ((lane >> 3) & 1) +
                    16 * ((4 * w_kk2 + 2 * (lane >> 5) + ((lane >> 4) & 1)) ^ turn(8 * w_d8));
  const int v_from = 4 * (2 * ((lane >> 3) & 1) + ((lane >> 4) & 1)) * DH + 8 * w_d8;
  // ROLE: 0 keys, 1 values, 2 both
  auto load_keys = [&](int i) KV_INLINE {
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const int row = (ws + x * SW) * KR;
      const int8_t* base = p.c.k_codes + place(k_at, 4 * i + (row >> 4)) + (row & 15) * DH;
      kraw[x] = *reinterpret_cast<const uint4*>(base + lane * 16);
    }
  };
  auto load_values = [&](int i) KV_INLINE {
    if (!has_v) return;
#pragma unroll
    for (int x = 0; x < VPER; ++x) {                        // piece x: 32 keys further
      const int64_t b0 = place(v_at, 4 * i + 2 * (w_kk2 + x)), b1 = place(v_at, 4 * i + 2 * (w_kk2 + x) + 1);
      const int8_t* base = p.c.v_codes + (lane >= 32 ? b1 : b0) + v_from;
#pragma unroll
      for (int e = 0; e < 4; ++e) vraw[x][e] = *reinterpret_cast<const uint2*>(base + e * DH);
    }
  };
  const uint32_t bias = 0x80808080u;
  auto store_keys = [&](int buf) KV_INLINE {
    const int at = k_put + buf * KBUF;
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      char* to = lds + x * SW * KR * DH * 2;
      const uint4 u = kraw[x];
      *reinterpret_cast<v8h*>(to + at) = code8(u.x ^ bias, u.y ^ bias);
      *reinterpret_cast<v8h*>(to + (at ^ 16)) = code8(u.z ^ bias, u.w ^ bias);
    }
  };
  auto store_values = [&](int buf) KV_INLINE {
    if (!has_v) return;
    const int at = v_put + buf * KBUF;
#pragma unroll
    for (int x = 0; x < VPER; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = (y ? vraw[x][e].y : vraw[x][e].x) ^ bias;
        // columns 0, 1 and 2, 3 of keys 0, 1 and of keys 2, 3
        const uint32_t l0 = __builtin_amdgcn_perm(a[1], a[0], 0x05010400u), l1 = __builtin_amdgcn_perm(a[3], a[2], 0x05010400u);
        const uint32_t h0 = __builtin_amdgcn_perm(a[1], a[0], 0x07030602u), h1 = __builtin_amdgcn_perm(a[3], a[2], 0x07030602u);
        const uint2 out[4] = {make_uint2(code_pair<kLow>(l0), code_pair<kLow>(l1)),
                              make_uint2(code_pair<kHigh>(l0), code_pair<kHigh>(l1)),
                              make_uint2(code_pair<kLow>(h0), code_pair<kLow>(h1)),
                              make_uint2(code_pair<kHigh>(h0), code_pair<kHigh>(h1))};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 4 * y + e;
          *reinterpret_cast<uint2*>(lds + (at ^ (64 * x) ^ (16 * c)) + 128 * c) = out[e];
        }
      }
  };

  float mref = -INFINITY, l = 0.0f, lref = -INFINITY;   // lref: log2 of vref
  // log2 of the weights' factor in a block with log2 sV of lv
  auto log_factor = [&](float lv) { return fmaxf(lv - (lref == -INFINITY ? 0.0f : lref), -60.0f) + 7.0f; };
  float lw = 0.0f, iw = 0.0f;                           // of cur's blocks while lref is one for all: that, its inverse
  auto factors = [&]() {
    lw = log_factor(cur.lv);
    iw = __builtin_amdgcn_exp2f(-lw);
  };
  factors();
  v16f acc[DB], s[2];
  v8h pw[4];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;

  const int k_get = n * DH * 2 + 16 * (g ^ (n & (PK >= 16 ? 15 : 7))), v_get = VBASE + n * 128 + 16 * (g ^ turn(n));
  auto values_product = [&](int buf) KV_INLINE {
    const int at = v_get + buf * KBUF;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const v8h a = *reinterpret_cast<const v8h*>(lds + (at ^ (32 * k) ^ (64 * (d & 1))) + 32 * 128 * d);
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, pw[k], acc[d], 0, 0, 0);
      }
  };
  auto keys_product = [&](int buf) KV_INLINE {
    const int at = k_get + buf * KBUF;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[k][e] = 0.0f;
#pragma unroll
    for (int x = 0; x < KS; ++x)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const v8h a = *reinterpret_cast<const v8h*>(lds + (at ^ (32 * x)) + 32 * DH * 2 * k);
        s[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, q[x], s[k], 0, 0, 0);
      }
  };
  // s[k][e]: key 32 k + 8 (e / 4) + 4 g + e % 4; blocks of 16 keys: e / 8 of s[k].
  // PARTLY: some of the wave's rows end before the tile does
  auto softmax = [&](int i, auto partly) KV_INLINE {
    constexpr bool PARTLY = decltype(partly)::value != 0;
    const int b0 = (4 * i) & 63;
    float top = lane_value(cur.lt, b0);                     // the largest lv of blocks with keys of the row
    const unsigned gone = static_cast<unsigned>(cur.gone >> b0) & 15u;
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = coef * lane_value(cur.sk, b0 + k);
    if (PARTLY || gone) {                                   // later keys, pages that are not there
      const int left = own_key - 64 * i - 4 * g;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int limit = (gone >> k) & 1 ? -1 : left;
        f[k] = fmaxf(f[k], 1e-37f);       // a page of scale 0: scores of about 0, not 0 * -inf
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (16 * k + 8 * (e / 4) + e % 4 > limit) s[k / 2][8 * (k & 1) + e] = -INFINITY;
      }
    }
    if constexpr (PARTLY) {
      top = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (16 * k <= own_key - 64 * i) top = fmaxf(top, lane_value(cur.lv, b0 + k));
    }
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float t = s[k / 2][8 * (k & 1)];
#pragma unroll
      for (int e = 1; e < 8; ++e) t = maximum(t, s[k / 2][8 * (k & 1) + e]);
      mx = maximum(mx, t * f[k]);
    }
    mx = pair_max(mx);
    if (__any(mx > mref + 8.0f || top > lref)) {
      const float m_new = fmaxf(mref, mx), l_new = fmaxf(lref, top);
      const float a = m_new > mref ? __builtin_amdgcn_exp2f(mref - m_new) : 1.0f;
      const float av = l_new > lref ? a * __builtin_amdgcn_exp2f(lref - l_new) : a;
      l *= a;
#pragma unroll
      for (int d = 0; d < DB; ++d) acc[d] *= av;
      mref = m_new;
      lref = l_new;
      factors();
    }
    const float base = mref == -INFINITY ? 0.0f : mref;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float c, inv;
      if constexpr (PARTLY) {
        c = log_factor(lane_value(cur.lv, b0 + k));         // of a block past the row: any finite value
        inv = __builtin_amdgcn_exp2f(-c);
      } else {
        c = lane_value(lw, b0 + k);
        inv = lane_value(iw, b0 + k);
      }
      c -= base;
      float t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t[e] = __builtin_amdgcn_exp2f(fmaf(s[k / 2][8 * (k & 1) + e], f[k], c));
        pw[k][e] = static_cast<_Float16>(t[e]);
      }
      l = fmaf(((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7])), inv, l);
    }
  };

  // the staging of matrix phase i; past the last tile it moves a page's codes
  // that nothing reads
  auto stage = [&](int i, auto role) KV_INLINE {
    constexpr int ROLE = decltype(role)::value;
    if constexpr (ROLE != 1) {
      store_keys(i & 1);                                    // of tile i + 2
      if (((i + 3) & 15) == 0) k_at = nxt.at;
      load_keys(i + 3);
    }
    if constexpr (ROLE != 0) {
      store_values((i + 1) & 1);
      if (((i + 2) & 15) == 0) v_at = nxt.at;
      load_values(i + 2);
    }
  };
  auto run = [&](auto role) KV_INLINE {
    constexpr int ROLE = decltype(role)::value;
    if constexpr (ROLE != 1) {
      load_keys(0);
      store_keys(0);
      load_keys(1);
      store_keys(1);
      load_keys(2);
    }
    if constexpr (ROLE != 0) {
      load_values(0);
      store_values(0);
      load_values(1);
    }
    lds_barrier();
    if (ROLE == 1) lds_barrier();                           // a phase behind
    if (active > 0) keys_product(0);
    lds_barrier();
    auto rotate = [&](int i) {                              // tile i + 1 opens a window
      if ((i + 1) & 15) return;
      cur = nxt;
      ++window;
      nxt = blocks(window + 1);
    };
    auto step = [&](int i, auto partly) KV_INLINE {
      softmax(i, partly);
#pragma unroll
      for (int k = 0; k < 4; ++k) {                         // all of it in this phase
        v4u whole = __builtin_bit_cast(v4u, pw[k]);
        asm volatile("" : "+v"(whole));
        pw[k] = __builtin_bit_cast(v8h, whole);
      }
      rotate(i);
      if (((i + 1) & 15) == 0) factors();
      lds_barrier();
      __builtin_amdgcn_s_setprio(2);
      stage(i, role);
      values_product(i & 1);
      keys_product((i + 1) & 1);                            // after the last tile: not used
      reads_ahead<4 * DB + 2 * KS>();
      __builtin_amdgcn_s_setprio(0);
      lds_barrier();
    };
    // A loop for the tiles that all of the wave's rows see to their end, and one for the
    // rest, where vref is a row's own (both by a branch in one loop: 187 instead of 175 us
    // for 4096 tokens and 32 heads)
    const int n_whole = min(active, (least_key + 1) / 64);
    for (int i = 0; i < n_whole; ++i) step(i, Int<0>{});
    for (int i = n_whole; i < active; ++i) step(i, Int<1>{});
    for (int i = active; i < n_tiles; ++i) {                // all of the wave's rows end before
      rotate(i);
      lds_barrier();
      stage(i, role);
      lds_barrier();
    }
    if (ROLE == 0) lds_barrier();
  };
  if (n_tiles > 0) {
    if (!TWO) run(Int<2>{});
    else if (w < SW) run(Int<0>{});
    else run(Int<1>{});
  }

  l += __shfl_xor(l, 32, 64);
  if (!live || (c0 > 0 && pos < c0)) return;
  const int64_t t = rq.t0 + tok;
  const int hq = h * group + hg;
  // the average of the codes, at most 2^7 times 127, before the values' scale
  const float unit = lref == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(lref - 7.0f);
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int d = 0; d < DB; ++d) acc[d] = acc[d] * inv * unit;
  if (pos < sp.chunk) {                   // the row's keys are all in this part
    // a lane pair holds columns 8 j + 4 g + 0..3: it trades halves, so that each
    // lane stores 8 columns in one piece
    uint16_t* o = p.out + t * p.ldo + static_cast<int64_t>(hq) * DH + 8 * g;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 8) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[i] = f32_to_bf16(acc[d][e + 2 * i]) | (static_cast<uint32_t>(f32_to_bf16(acc[d][e + 2 * i + 1])) << 16);
        const auto x = __builtin_amdgcn_permlane32_swap(u[0], u[2], false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(u[1], u[3], false, false);
        *reinterpret_cast<uint4*>(o + 32 * d + 2 * e) = make_uint4(x[0], y[0], x[1], y[1]);
      }
  } else {
    const int64_t at = (sp.row(b, tok, t) * p.Hq + hq) * sp.parts + part;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4*>(sp.o + at * DH + 32 * d + 2 * e + 4 * g) =
            make_float4(acc[d][e], acc[d][e + 1], acc[d][e + 2], acc[d][e + 3]);
    if (g == 0) sp.ml[at] = make_float2(mref, l);
  }
}

// Joins the parts of rows that span more than one: o = sum_s g_s o_s, g_s = 2^(m_s - m)
// l_s / sum_s 2^(m_s - m) l_s, kept as an average all the way, by WPR waves per row: 4 where there are more than 8 parts and
// at most 1024 rows, else 1 (a call with 32 parts of 256 keys 11.4 us with 4 and 12.5
// with 1, with 16 14.9 and 15.4, with 8 and fewer the same; 2048 rows of up to 9 parts
// 7.4 us and 5.4). Bound by latency: the parts' maxima,
// then eight loads at a time; about 4 us of a call that is split. TOKENS: rows are
// counted over the batch (for requests of many rows), over both dimensions of the
// grid, as one holds fewer than 2^32 threads; else over a request, blockIdx.y (one
// lookup less before the parts can be asked for).
template <int DH, int WPR, bool TOKENS>
__global__ __launch_bounds__(256) void combine_kernel(KvAttnArgs p, Split sp) {
  constexpr int C = DH / 64;
  __shared__ float o_s[4][DH];
  __shared__ float l_s[4], m_s[4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, part0 = w % WPR;
  const int block = TOKENS ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x;
  const int row = block * (4 / WPR) + w / WPR, hq = row % p.Hq;   // < 2^30 + 2^22
  int tok = row / p.Hq, b = blockIdx.y;
  if (TOKENS) b = wave_search(static_cast<int>(p.B), tok, [&](int i) { return static_cast<int64_t>(max(p.cu_new[i], 0)); });
  const Request rq = request(p, b);
  if (TOKENS) tok -= rq.t0;
  const int rows = rq.tokens * (p.Hq / p.c.H);
  const int64_t at_pos = rq.first_pos + tok;
  const int64_t chunk = TOKENS ? sp.chunk : sp.part_keys(rq.first_pos + rq.tokens);
  // the same for all waves of a row; a row without parts to join stays out
  const bool join = tok >= 0 && tok < rq.tokens && rows > sp.least_rows && rows <= sp.most_rows &&
                    at_pos >= chunk;
  if (WPR == 4 && !join) return;
  const int n = join ? static_cast<int>(static_cast<uint32_t>(at_pos) / static_cast<uint32_t>(chunk)) + 1 : 0;
  const int64_t base = (sp.row(b, tok, rq.t0 + tok) * p.Hq + hq) * sp.parts;
  const int per = (n + WPR - 1) / WPR, s0 = min(part0 * per, n), s1 = min(s0 + per, n);
  float top = -INFINITY, sum = 0.0f, o[C] = {};
  for (int s = s0; s < s1; s += 64) {
    const int k = min(64, s1 - s);
    const float2 ml = lane < k ? sp.ml[base + s + lane] : make_float2(-INFINITY, 0.0f);
    const float t = fmaxf(top, wave_max(ml.x));
    if (t == -INFINITY) continue;
    const float before = top == -INFINITY ? 0.0f : sum * __builtin_amdgcn_exp2f(top - t);
    const float mass = ml.x == -INFINITY ? 0.0f : ml.y * __builtin_amdgcn_exp2f(ml.x - t);
    top = t;
    float x = mass;
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
    sum = before + x;
    const float inv = __builtin_amdgcn_rcpf(sum), f = mass * inv, keep = before * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= keep;
    for (int i = 0; i < k; i += 8) {   // eight loads in flight; past k the last part again, with weight 0
      float src[8][C];
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int c = 0; c < C; ++c) src[u][c] = sp.o[(base + s + min(i + u, k - 1)) * DH + C * lane + c];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float fu = i + u < k ? lane_value(f, i + u) : 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = fmaf(fu, src[u][c], o[c]);
      }
    }
  }
  if (lane == 0) {
    m_s[w] = top;
    l_s[w] = sum;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) o_s[w][C * lane + c] = o[c];
  __syncthreads();
  if (!join || part0 != 0 || lane >= DH / 8) return;
  float all = -INFINITY, total = 0.0f, v[8] = {};
#pragma unroll
  for (int u = 0; u < WPR; ++u) all = fmaxf(all, m_s[w + u]);
#pragma unroll
  for (int u = 0; u < WPR; ++u)
    total += m_s[w + u] == -INFINITY ? 0.0f : l_s[w + u] * __builtin_amdgcn_exp2f(m_s[w + u] - all);
  const float inv = total > 0.0f ? __builtin_amdgcn_rcpf(total) : 0.0f;
#pragma unroll
  for (int u = 0; u < WPR; ++u) {
    const float f = m_s[w + u] == -INFINITY ? 0.0f : l_s[w + u] * __builtin_amdgcn_exp2f(m_s[w + u] - all) * inv;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(f, o_s[w + u][8 * lane + i], v[i]);
  }
  store_row8(p, rq.t0 + tok, hq, 8 * lane, v);
}

// ---------------------------------------------------------------- host
// How a call is run: requests of at most `few` rows by the split kernel with
// NC tiles of 16 rows (few = 16 NC; NC = 0: none), others by the tile kernel.
struct Config {
  int NC = 0;
  bool tiles = false;
  int64_t chunk[2] = {0, 0};    // keys of a part: split kernel, tile kernel
  int parts[2] = {1, 1};
  int items = 0;                // row tiles of the tile kernel, at most
  int64_t part_rows[2] = {0, 0};   // tokens whose parts are kept
  int tokens = 0, least = 0;    // see Split
};

constexpr int tile_waves(int64_t dh) { return dh == 256 ? 4 : 8; }
constexpr int kSplitWaves = 4;

void cut(int64_t max_kv, int64_t chunk, int64_t& c, int& parts) {
  c = chunk;
  parts = static_cast<int>(std::max<int64_t>((max_kv + chunk - 1) / chunk, 1));
}

// Parts of the tile kernel's keys, for `groups` workgroups a part and `rows` rows and
// heads: the least of an estimate in microseconds. A tile of 64 keys takes 2.2 (1.2
// for dh = 64, 3 for 256), a workgroup's start and end about three tiles, its averages
// three more; the join is 4 and the averages, written and read at 5 TB/s. The 256 CUs
// of the card (one number, so that the workspace's size is the same for every caller)
// take the workgroups in whole rounds, if those are alike (one request); those of
// several requests, whose lengths may differ, fill the last round in part.
// Over 85 calls of one to six requests with 16 to 1000 workgroups, each with every
// number of parts up to 8 (32 for one request), the estimate's choice is 2.8% off the
// best in the mean: 0.5% where 256 to 511 workgroups take the keys of several requests
// (two prompts of 1500, 32 query and 8 key heads of 128: one part 61 us, two 111; three
// of 1111 after 12000: 735 and 828; of 1111, 601 and 717 after 12000, 4845 and 2214:
// two parts 399, one 414, four 403, with parts of 4480 keys 389), 2.3% for one request
// (512 tokens after 8192 keys: four parts 96, three 107, two 140, eight 110, one 232;
// 4096 tokens, 32 heads: one 162, two 213), 14% for several that leave CUs without work.
void tile_parts(int64_t groups, bool equal, int64_t rows, int64_t dh, int64_t max_kv, int64_t& chunk,
                int& parts) {
  const double tile_us = dh == 64 ? 1.2 : dh == 128 ? 2.2 : 3.0;
  double best = 0.0;
  for (int64_t n = 1; n == 1 || (n <= 64 && n * 256 <= max_kv); ++n) {
    const int64_t tiles = (max_kv + 64 * n - 1) / (64 * n);
    const double full = static_cast<double>(groups * n) / 256.0, whole = std::ceil(full);
    const double rounds = equal ? whole : 0.25 * whole + 0.75 * full + 0.5;
    const double join = n > 1 ? 4.0 + static_cast<double>(rows * n * dh) * 8.0 / 5.0e6 : 0.0;
    const double us = rounds * static_cast<double>(tiles + (n > 1 ? 6 : 3)) * tile_us + join;
    if (n > 1 && us >= 0.97 * best) continue;
    best = us;
    cut(max_kv, std::max<int64_t>(64 * tiles, 64), chunk, parts);
  }
}

Config config(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t dh, int64_t max_new, int64_t max_kv) {
  Config c;
  const int64_t group = Hq / H, most = std::min(max_new, T), rows = most * group;
  // Rows that the split kernel takes, against the tile kernel with parts of its own,
  // of which a wave has 32 rows and a workgroup 256 (8 key heads, 4096 keys each; one
  // request, 8 and 64). 64 rows of 64: 17, 32, 141 us and 16, 32, 151; 48 of 128: 21,
  // 37, 170 and 20, 38, 286; 32 of 128: 16, 29, 143 and 19, 36, 189; 32 of 256: 27, 59,
  // 363 and 32, 66, 387. 64 of 128 would spill registers: 24, 47, 227 and 21, 39, 196. A
  // form for more rows at 16 of 128: 27 instead of 22 us for 8 requests.
  const int64_t few = dh == 256 ? 32 : dh == 128 ? 48 : 64;
  int64_t apart = 0;            // requests of few rows beside longer ones
  c.tiles = rows > few;
  if (!c.tiles) c.NC = rows <= 16 ? 1 : rows <= 32 ? 2 : dh == 128 ? 3 : 4;
  // Unequal requests: those of few rows apart, by two more launches, if they can be
  // so many (T rows are in B requests of at most `most`) or so long that it pays:
  // with a prompt of 512 tokens, 8 key heads of 128, 8 single tokens at 4096 keys
  // take 53 us apart and 58 in the tile kernel, 15: 60 and 85, 2 at 16384: 55 and 99,
  // one at 8192, the prompt too: 112 and 135; but 4 at 4096: 47 and 37, 16 at 1000: 48
  // and 39.
  else if (group <= 16) {
    apart = std::min(std::max<int64_t>(B * most - T, 0) / (most - 16 / group), B - 1);
    if (apart > 0 && (max_kv >= 8192 || apart * max_kv * H >= 1 << 18)) c.NC = 1;
  }
  if (c.NC) {
    // About one workgroup for each CU (of 256): its four waves keep 32 KiB on
    // their way, and there is little to join. With two: 28.1 instead of 27.2 us for
    // 8 requests of up to 2048 keys and 32 heads, 61.3 instead of 59.4 us for one
    // request of 131072 keys and 8 heads; with four 32.4 and 63.4. But at most 2048 keys
    // where there are several requests, whose lengths may differ (4096: 64 of 100 to
    // 15951 keys, 509000 in all, 8 heads, 216 instead of 207 us, 32 of 10 to 8088, 128000
    // in all, 64 instead of 56; eight of 16384 each beside a prompt 67 instead of 75), up
    // to 4096 keys without a split (63 of 4096 beside a prompt 176, in two parts 192), and
    // no more than 8192 workgroups, as those that a long bound leaves empty take a
    // nanosecond each (64 of 1000 keys, bound 131072: 49 us with 32768, 35 with 16384);
    // else at most the 4096 that the lanes hold the pages of.
    // A request's own parts follow its length, not the bound (see part_keys), in parts
    // of no less than 4 keys for each request and head, which fill the CUs without a
    // split: with a bound of 131072 keys one request of 4000 takes 11.6 us (41 with the
    // bound's parts), 64 of 1000 35 us (27 with a bound of 1001).
    constexpr int64_t NW = kSplitWaves, unit = 32 * NW;
    const int64_t want = (max_kv * B * H + 255) / 256, half = 512 * NW;
    const bool finer = B > 1 && max_kv > 2 * half && (max_kv + half - 1) / half * B * H <= 8192;
    cut(max_kv, std::min(std::max<int64_t>((want + unit - 1) / unit * unit, 256), finer ? half : 2 * half),
        c.chunk[0], c.parts[0]);
    static_assert(32 * kSplitWaves == Split::unit, "a tile of 32 keys for each wave");
    c.least = static_cast<int>(std::min<int64_t>(std::max<int64_t>((B * H + 31) / 32 * unit, 256), c.chunk[0]));
    // the parts of the few-row requests alone, where that is less
    const int64_t tokens = std::min(most, 16 * c.NC / group);
    if (B * tokens < T) c.tokens = static_cast<int>(tokens);
    c.part_rows[0] = std::min(B * tokens, T);
  }
  if (c.tiles) {
    c.part_rows[1] = T;
    const int64_t tile = 32 * tile_waves(dh);
    c.items = static_cast<int>(T * group / tile + B);
    const int64_t longer = B - apart;
    const int64_t groups = H * std::min(std::max<int64_t>(T - apart, 1) * group / tile + longer,
                                        longer * ((rows + tile - 1) / tile));
    tile_parts(groups, longer == 1, T * Hq, dh, max_kv, c.chunk[1], c.parts[1]);
  }
  return c;
}

// bytes of the parts of the split kernel (0) or the tile kernel (1)
size_t part_bytes(const Config& c, int i, int64_t Hq, int64_t dh) {
  return c.parts[i] < 2 ? 0 : (static_cast<size_t>(c.part_rows[i]) * Hq * c.parts[i] * (dh + 2) * sizeof(float) + 255) / 256 * 256;
}

Split parts_at(void* ws, const KvAttnArgs& a, const Config& c, int i, int least, int most) {
  Split sp{nullptr, nullptr, c.chunk[i], c.parts[i], least, most, i == 0 ? c.tokens : 0, c.least};
  if (sp.parts > 1) {
    sp.o = static_cast<float*>(ws);
    sp.ml = reinterpret_cast<float2*>(sp.o + c.part_rows[i] * a.Hq * sp.parts * a.c.dh);
  }
  return sp;
}

template <int DH, int WPR, bool TOKENS>
void launch_combine_rows(const KvAttnArgs& a, const Split& sp, int64_t rows, int64_t requests, hipStream_t s) {
  const int64_t blocks = (rows * WPR + 3) / 4, wide = std::min<int64_t>(blocks, 1 << 20);
  const dim3 grid(static_cast<unsigned>(TOKENS ? wide : blocks),
                  static_cast<unsigned>(TOKENS ? (blocks + wide - 1) / wide : requests));
  combine_kernel<DH, WPR, TOKENS><<<grid, 256, 0, s>>>(a, sp);
}

template <int DH, bool TOKENS>
void launch_combine(const KvAttnArgs& a, const Split& sp, hipStream_t s) {
  if (sp.parts < 2) return;
  // of each request, at most the tokens that make most_rows rows; or all of the batch
  const int64_t few = std::min(std::min(a.max_new, a.T), static_cast<int64_t>(sp.most_rows) * a.c.H / a.Hq);
  const int64_t rows = (TOKENS ? a.T : few) * a.Hq, requests = TOKENS ? 1 : a.B;
  if (sp.parts > 8 && rows * requests <= 1024) launch_combine_rows<DH, 4, TOKENS>(a, sp, rows, requests, s);
  else launch_combine_rows<DH, 1, TOKENS>(a, sp, rows, requests, s);
}

// more LDS than the 64 KiB that a kernel may use unasked
template <class K>
hipError_t allow_lds(K kernel, int bytes) {
  return bytes <= 65536 ? hipSuccess
                        : hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                              hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int DH, int NC>
hipError_t launch_split(const KvAttnArgs& a, const Split& sp, hipStream_t s) {
  constexpr int NW = kSplitWaves, lds = NW * 16 * NC * (DH + 6) * static_cast<int>(sizeof(float));
  const hipError_t e = allow_lds(split_kernel<DH, NC, NW>, lds);
  if (e != hipSuccess) return e;
  // Parts come last: workgroups go to the 8 XCDs in turn, and with the parts first
  // those of short requests under a long bound, all but the first of them empty, would
  // share few XCDs.
  const dim3 grid(a.c.H, static_cast<unsigned>(a.B), sp.parts);
  split_kernel<DH, NC, NW><<<grid, 64 * NW, lds, s>>>(a, sp);
  launch_combine<DH, false>(a, sp, s);
  return hipSuccess;
}

template <int DH>
hipError_t launch_dh(const KvAttnArgs& a, const Config& c, void* ws, hipStream_t s) {
  if (c.NC) {
    const Split sp = parts_at(ws, a, c, 0, 0, 16 * c.NC);
    const hipError_t e = c.NC == 1   ? launch_split<DH, 1>(a, sp, s)
                         : c.NC == 2 ? launch_split<DH, 2>(a, sp, s)
                                     : launch_split<DH, DH == 64 ? 4 : DH == 128 ? 3 : 2>(a, sp, s);
    if (e != hipSuccess) return e;
  }
  if (c.tiles) {
    constexpr int NW = tile_waves(DH), lds = 2 * 2 * 64 * DH * 2;
    const hipError_t e = allow_lds(tile_kernel<DH, NW>, lds);   // 128 KiB for DH = 256
    if (e != hipSuccess) return e;
    const Split sp = parts_at(static_cast<uint8_t*>(ws) + part_bytes(c, 0, a.Hq, DH), a, c, 1, 16 * c.NC,
                              0x7fffffff);
    const dim3 grid(static_cast<unsigned>(c.items) * a.c.H, sp.parts);
    tile_kernel<DH, NW><<<grid, 64 * NW, lds, s>>>(a, sp, c.items);
    launch_combine<DH, true>(a, sp, s);
  }
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t dh,
                              int64_t max_new, int64_t max_kv) {
  const Config c = config(T, B, Hq, H, dh, max_new, max_kv);
  return part_bytes(c, 0, Hq, dh) + part_bytes(c, 1, Hq, dh);
}

hipError_t launch_kv_attention(const KvAttnArgs& a, void* ws, hipStream_t s) {
  const Config c = config(a.T, a.B, a.Hq, a.c.H, a.c.dh, a.max_new, a.max_kv);
  return a.c.dh == 64 ? launch_dh<64>(a, c, ws, s) : a.c.dh == 128 ? launch_dh<128>(a, c, ws, s)
                                                                   : launch_dh<256>(a, c, ws, s);
}

}  // namespace rw4

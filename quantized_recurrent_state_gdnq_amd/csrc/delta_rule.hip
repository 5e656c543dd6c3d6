// The gated delta rule with its state in fp32: chunks of 64 tokens on the
// matrix units (forward), and one token per sequence.  The backward pass is in
// delta_rule_backward.hip; the formulas are in delta_common.h.
#include <type_traits>

#include "delta_common.h"
#include "delta_prep.h"

namespace gdnq {
namespace {

// ---------------------------------------------------------------- the chain
//
// A workgroup of four waves takes 64 rows (d_v) of one head's state through
// its chunks, 16 rows a wave, in registers as S^T in tiles of 16 columns (d_k)
// x 16 rows.  No wave needs another's results: the second operand of every
// product is the wave's own (see chain_row), the first ones (K, Q and the
// triangles) come from LDS, where the workgroup puts the next chunk's while
// this one's are used: its loads are made between this chunk's products, its
// operands read from LDS some products ahead of their own.
//   Bound by one wave a SIMD: a chunk is 176 matrix instructions of 16 cycles and
// about 900 others in a chain of products of which each needs the one before, 3.4
// us a chunk of 128 x 128; with SAVE (96 KB more to store a chunk and head) 4.6.
// 4 x 8192 tokens, 16 heads: 434 us, 755 MB of memory at 1.7 TB/s, with half of the
// CUs idle: there are no more rows, and segments would be 1.9 times the work.  The
// third part of S, x and w is 44 of the products and 70 of the microseconds: without
// it the state is 4e-6 of its norm off, with it 1e-6.
//   SAVE: S and w of every chunk are left in the carry.
//   PASS: the first pass over segments, which has no outputs.
template <int DK, bool SAVE, bool PASS, typename O>
__global__ __launch_bounds__(256, PASS ? 2 : 1) void delta_chain_kernel(DeltaLaunch L, int row_groups) {
  constexpr int KB = DK / 32, TILES = DK / 16, P = PASS ? 2 : 3;  // parts of what passes on
  using Loader = ChainLoader<DK, false>;
  using Buffer = ChainBuffer<DK, false, PASS>;
  __shared__ __attribute__((aligned(1024))) Buffer buffers[2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  int within;
  const int unit = xcd_unit(row_groups * (L.H / L.G), within);
  const DeltaItem item = delta_item(L, unit / L.G, PASS);
  if (item.b < 0) return;
  const int b = item.b;
  const DeltaSpan s = delta_sequence(L, b);
  const int chunks = (s.tokens + 63) / 64;
  const ChainPlace place = chain_place(L, row_groups, chunks, item, unit % L.G, within);
  const int h = place.h, group = place.group, end = place.end;
  const int col = group * 64 + wave * 16 + c;
  const bool mine = col < L.dv;
  Loader loader;
  loader.init(L, L.v, h, PASS && place.identity ? 0 : group, wave, lane);
  const int64_t vrow = int64_t(L.H) * L.dv;
  const int tiles = (L.dk + 31) / 32 * 2;  // of a row of the state that it leaves
  const bool exact = L.dk == DK && group * 64 + wave * 16 + 16 <= L.dv;  // all lanes leave something

  f32x4 S[TILES];
  const int64_t state_row = ((int64_t(b) * L.H + h) * L.dv + col) * L.dk;
  if constexpr (PASS) {
    if (place.identity)
      chain_identity<TILES>(S, col, g);
    else
      chain_load_state<TILES>(S, nullptr, L.dk, col, mine, g);
  } else {
    const float* start = L.h0 ? L.h0 + state_row - int64_t(col) * L.dk : nullptr;
    if (item.seg > 0) start = reinterpret_cast<const float*>(delta_segment(L, int(item.at) + item.seg - 1, h));
    chain_load_state<TILES>(S, start, L.dk, col, mine, g);
  }
  loader.clear(buffers[0]);
  loader.clear(buffers[1]);
  if (place.first < end)
    loader.template load<false, PASS>(buffers[place.first & 1], loader.next(s.first + int64_t(place.first) * 64,
                                                                     min(64, s.tokens - place.first * 64), s.slot + place.first));
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  for (int chunk = place.first; chunk < end; ++chunk) {
    const Buffer& buf = buffers[chunk & 1];
    const int64_t first = s.first + int64_t(chunk) * 64;
    const int n = min(64, s.tokens - chunk * 64);
    Buffer& following = buffers[(chunk + 1) & 1];
    const auto next = loader.next(first + 64, min(64, s.tokens - chunk * 64 - 64), s.slot + chunk + 1);
    const bool paced = chunk + 1 < end && next.whole;
    if (chunk + 1 < end && !next.whole) loader.template load<false, PASS>(following, next);
    auto ahead = [&](auto step) {
      phase();
      if (paced) loader.template step<step.value, PASS>(following, next);
    };
    float* left = nullptr;  // this chunk's part of the carry
    if constexpr (SAVE)
      left = reinterpret_cast<float*>(static_cast<uint8_t*>(L.carry) + ((s.slot + chunk) * L.H + h) * delta_left_bytes(L));
    // K, then Q, 32 columns at a time, two ahead
    bf16x8 ring[3][4];
    const uint8_t* queries = nullptr;
    if constexpr (!PASS) queries = buf.q;
    auto read = [&](auto i) { chain_rows<DK>(i.value < KB ? buf.k : queries, lane, i.value % KB, ring[i.value % 3]); };
    read(Int<0>{});
    read(Int<1>{});
    phase();
    bf16x8 sp[KB][P];
#pragma unroll
    for (int j = 0; j < KB; ++j) split8(S[2 * j], S[2 * j + 1], sp[j]);
    const float* rows = reinterpret_cast<const float*>(buf.rows);
    auto row4 = [&](int which, int it) { return *reinterpret_cast<const f32x4*>(rows + which * 64 + chain_row(it, g * 4)); };
    phase();
    // x = V - c K S^T by tokens (rows), and O^T = (c Q S^T)^T by tokens in lanes,
    // so that a lane has four adjacent values of a token to store: the operands
    // are the same registers, in the other order.
    f32x4 x[4] = {}, o[4] = {}, decay[4];
    s16x4 v[4];
    bf16x8 xp[2][P], n2[2][TRI_BLOCKS];
    auto errors = [&](auto half) {
#pragma unroll
      for (int it = 2 * half.value; it < 2 * half.value + 2; ++it)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float value = PASS && place.identity ? 0.0f : bf16_value(v[it][e]);
          x[it][e] = value - decay[it][e] * x[it][e];
        }
      split8(x[2 * half.value], x[2 * half.value + 1], xp[half.value]);
    };
    // A quarter of the state that enters; behind the last load, so that the wait for
    // the loads need not wait for these stores too.
    auto leave = [&](auto quarter) {
      phase();
      if constexpr (SAVE) {
#pragma unroll
        for (int t = quarter.value * (TILES / 4); t < (quarter.value + 1) * (TILES / 4); ++t) {
          float* to = left + left_place(col, t, tiles, g);
          if (exact || (mine && chain_row(t, g * 4) < L.dk)) *reinterpret_cast<f32x4*>(to) = S[t];
        }
        phase();
      }
    };
    constexpr int PRODUCTS = PASS ? KB : 2 * KB, STEPS = Loader::STEPS;
    each<PRODUCTS>([&](auto i) {
      constexpr int j = i.value % KB;
      if constexpr (i.value + 2 < PRODUCTS) read(Int<i.value + 2>{});
      if constexpr (i.value == (PASS ? KB - 2 : KB - 1)) {
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          v[it] = chain_column(buf.v, it, wave, lane);
          decay[it] = row4(ROW_C, it);
        }
      }
      if constexpr (i.value == PRODUCTS - 2) chain_triangle(buf.tri, lane, n2);
      phase();
      const bf16x8(&f)[4] = ring[i.value % 3];
      if constexpr (i.value < KB) {
#pragma unroll
        for (int p = P - 1; p >= 0; --p)
#pragma unroll
          for (int it = 0; it < 4; ++it) x[it] = mfma16(f[it], sp[j][p], x[it]);
      } else {
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
          for (int it = 0; it < 4; ++it) o[it] = mfma16(sp[j][p], f[it], o[it]);
      }
      if constexpr (!PASS && i.value >= 2 * KB - 2) errors(Int<i.value - (2 * KB - 2)>{});  // beside the last of these products
      each<STEPS>([&](auto s) {
        if constexpr (s.value * PRODUCTS / STEPS == i.value) ahead(s);
      });
    });
    if constexpr (PASS) {
      errors(Int<0>{});
      errors(Int<1>{});
    }
    phase();
    bf16x8 kt[2][4][2];
    chain_columns<DK>(buf.k, lane, 0, kt[0]);
    f32x4 tail[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) tail[it] = row4(ROW_TAIL_BETA, it);
    const float whole = rows[ROW_C * 64 + 63];
    float decay_o[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) decay_o[it] = rows[ROW_C * 64 + chain_row(it, c)];
    phase();
    // The six blocks of a triangle: tiles 0 and 1 with the first 32 tokens, 2 and
    // 3 with both halves.
    f32x4 w[4] = {};
    part_terms<2, P>([&](auto i, auto j) {
      const bf16x8(&n)[TRI_BLOCKS] = n2[i.value];
#pragma unroll
      for (int it = 0; it < 4; ++it) w[it] = mfma16(n[it < 2 ? it : 2 * it - 2], xp[0][j.value], w[it]);
#pragma unroll
      for (int it = 2; it < 4; ++it) w[it] = mfma16(n[2 * it - 1], xp[1][j.value], w[it]);
      if constexpr (SAVE && i.value == 0 && j.value > 0) {  // beside the products
        leave(Int<(P - 1 - j.value) * 2>{});
        leave(Int<(P - 1 - j.value) * 2 + 1>{});
      }
    });
#pragma unroll
    for (int t = 0; t < TILES; ++t) S[t] *= whole;
#pragma unroll
    for (int it = 0; it < 4; ++it) o[it] *= decay_o[it];
    phase();
    bf16x8 m2[2][TRI_BLOCKS], tp[2][P], wp[2][2];
    if constexpr (TILES > 4) chain_columns<DK>(buf.k, lane, 1, kt[1]);
    if constexpr (!PASS) chain_triangle(buf.tri + TRI_BYTES, lane, m2);
    phase();
#pragma unroll
    for (int j = 0; j < 2; ++j) split8(w[2 * j] * tail[2 * j], w[2 * j + 1] * tail[2 * j + 1], tp[j]);
    chain_update(S, kt[0], tp);
    if constexpr (!PASS) {
#pragma unroll
      for (int j = 0; j < 2; ++j) split8(w[2 * j], w[2 * j + 1], wp[j]);
    }
    phase();
    if constexpr (TILES > 4) chain_update(S + 4, kt[1], tp);
    phase();
    if constexpr (!PASS)
      part_terms<2, 2>([&](auto i, auto j) {
        const bf16x8(&m)[TRI_BLOCKS] = m2[i.value];
#pragma unroll
        for (int it = 0; it < 4; ++it) o[it] = mfma16(wp[0][j.value], m[it < 2 ? it : 2 * it - 2], o[it]);
#pragma unroll
        for (int it = 2; it < 4; ++it) o[it] = mfma16(wp[1][j.value], m[2 * it - 1], o[it]);
      });
    phase();
    // the next chunk is in LDS, and nobody reads this one any more; the stores
    // below are behind this wait, so that the next chunk's covers them
    if (SAVE && exact)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(TILES) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if constexpr (SAVE) {
      if (mine) {
        float* to = left + delta_state_floats(L);
#pragma unroll
        for (int it = 0; it < 4; ++it) *reinterpret_cast<f32x4*>(to + left_place(col, it, 4, g)) = w[it];
      }
    }
    const int oc = group * 64 + wave * 16 + g * 4;
    if (!PASS && oc < L.dv) {
      O* op = static_cast<O*>(L.o) + first * vrow + int64_t(h) * L.dv + oc;
      typedef O o4 __attribute__((ext_vector_type(4)));
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int row = chain_row(it, c);
        if (row < n) *reinterpret_cast<o4*>(op + row * vrow) = __builtin_convertvector(o[it], o4);
      }
    }
  }
  if constexpr (PASS) chain_leave<TILES>(L, item, place, S, col, g);
  if (!PASS && L.h_last && mine && end == chunks) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int at = chain_row(t, g * 4);
      if (at < L.dk) *reinterpret_cast<f32x4*>(L.h_last + state_row + at) = S[t];
    }
  }
}

// ---------------------------------------------------------------- one token
//
// Bound by the state's bytes: read once, written once (64 sequences, 32 heads of 128 x
// 128: 51.5 us, 5.29 TB/s; one sequence of 16 heads: 3.5 us, the launch).  LANES lanes hold a row,
// eight columns each, and R rows are in flight in a lane.
template <int LANES, int R, typename E>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaLaunch L) {
  constexpr int ROWS = 256 / LANES;  // rows of a pass
  const int lane = threadIdx.x % LANES, at = lane * 8;
  const bool here = at < L.dk;
  const int row0 = blockIdx.x % L.row_groups * (ROWS * R) + threadIdx.x / LANES;
  const int64_t bh = blockIdx.x / L.row_groups;
  const int h = int(bh % L.H);
  const int64_t b = bh / L.H, key = (b * L.G + h / (L.H / L.G)) * L.dk + at;
  const float* from = L.h0 + bh * L.dv * L.dk + at;
  float* to = L.h_last + bh * L.dv * L.dk + at;
  f32x4 s[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + r * ROWS;
    s[r][0] = s[r][1] = f32x4{0, 0, 0, 0};
    if (here && row < L.dv) {
      s[r][0] = *reinterpret_cast<const f32x4*>(from + int64_t(row) * L.dk);
      s[r][1] = *reinterpret_cast<const f32x4*>(from + int64_t(row) * L.dk + 4);
    }
  }
  float k[8] = {}, q[8] = {};
  if (here) {
    const E* kp = static_cast<const E*>(L.k) + key;
    const E* qp = static_cast<const E*>(L.q) + key;
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = to_f32(kp[e]), q[e] = to_f32(qp[e]);
  }
  float kq = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) kq = fmaf(k[e], q[e], kq);
  kq = group_sum<LANES>(kq);
  float a = L.alpha[bh];
  if (L.log_decay) a = expf(a);
  const float beta = L.beta[bh];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + r * ROWS;
    float sk = 0, sq = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = s[r][e / 4][e % 4] * a;
      s[r][e / 4][e % 4] = x;
      sk = fmaf(x, k[e], sk);
      sq = fmaf(x, q[e], sq);
    }
    sk = group_sum<LANES>(sk);
    sq = group_sum<LANES>(sq);
    if (row < L.dv) {
      const float u = beta * (to_f32(static_cast<const E*>(L.v)[bh * L.dv + row]) - sk);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[r][e / 4][e % 4] = fmaf(u, k[e], s[r][e / 4][e % 4]);
      if (here) {
        *reinterpret_cast<f32x4*>(to + int64_t(row) * L.dk) = s[r][0];
        *reinterpret_cast<f32x4*>(to + int64_t(row) * L.dk + 4) = s[r][1];
      }
      if (lane == 0) {
        const float o = fmaf(u, kq, sq);
        if (L.out_bf16)
          store_f32(static_cast<bf16*>(L.o) + bh * L.dv + row, o);
        else
          store_f32(static_cast<float*>(L.o) + bh * L.dv + row, o);
      }
    }
  }
}

template <int DK>
hipError_t forward(const DeltaLaunch& L, hipStream_t stream) {
  const int64_t heads = delta_slots(L) * L.H;
  if (heads > 0) {
    delta_prep_kernel<DK, false><<<uint32_t(heads), 256, 0, stream>>>(L);
    if (hipError_t e = hipGetLastError()) return e;
  }
  const int groups = (L.dv + 63) / 64;
  if (L.segments > 1) {
    const int all = groups + (L.dk + 63) / 64;
    delta_chain_kernel<DK, false, true, bf16><<<uint32_t(all * L.H * delta_items(L, true)), 256, 0, stream>>>(L, all);
    if (hipError_t e = hipGetLastError()) return e;
    delta_join_kernel<DK, false><<<uint32_t(groups * L.H * L.B), 256, 0, stream>>>(L, groups);
    if (hipError_t e = hipGetLastError()) return e;
  }
  const uint32_t grid = uint32_t(groups * L.H * delta_items(L, false));
  if (L.carry)
    L.out_bf16 ? delta_chain_kernel<DK, true, false, bf16><<<grid, 256, 0, stream>>>(L, groups)
               : delta_chain_kernel<DK, true, false, float><<<grid, 256, 0, stream>>>(L, groups);
  else
    L.out_bf16 ? delta_chain_kernel<DK, false, false, bf16><<<grid, 256, 0, stream>>>(L, groups)
               : delta_chain_kernel<DK, false, false, float><<<grid, 256, 0, stream>>>(L, groups);
  return hipGetLastError();
}

// Four rows a lane where that still is 1024 workgroups, four a CU, else one (us with
// four rows, with one; 128 x 128 unless said): 256 workgroups of four rows 6.7, 6.3; 512
// 10.2, 9.7; 768 14.0, 14.8; 1024 15.8, 17.6 (64 x 64 9.9, 9.7; 256 x 256 15.4, 17.4); 4096
// 52.4, 55.4.
template <int LANES, typename E>
hipError_t step(DeltaLaunch L, hipStream_t stream) {
  constexpr int ROWS = 256 / LANES;
  auto groups = [&](int r) { return (L.dv + ROWS * r - 1) / (ROWS * r); };
  const int64_t heads = int64_t(L.B) * L.H;
  if (heads * groups(4) >= 1024) {
    L.row_groups = groups(4);
    delta_step_kernel<LANES, 4, E><<<uint32_t(heads * L.row_groups), 256, 0, stream>>>(L);
  } else {
    L.row_groups = groups(1);
    delta_step_kernel<LANES, 1, E><<<uint32_t(heads * L.row_groups), 256, 0, stream>>>(L);
  }
  return hipGetLastError();
}

template <typename E>
hipError_t step_of(const DeltaLaunch& L, hipStream_t stream) {
  if (L.dk <= 64) return step<8, E>(L, stream);
  if (L.dk <= 128) return step<16, E>(L, stream);
  return step<32, E>(L, stream);
}

}  // namespace

size_t delta_carry_bytes(const DeltaLaunch& L) { return size_t(delta_slots(L)) * L.H * delta_left_bytes(L); }
static DeltaLaunch forward_split(DeltaLaunch L) {
  delta_split(L, delta_slots(L) * L.H * delta_chunk_bytes(false));
  return L;
}
size_t delta_forward_workspace_bytes(const DeltaLaunch& L) { return size_t(delta_split_bytes(forward_split(L))); }

hipError_t launch_delta_forward(const DeltaLaunch& L, hipStream_t stream) {
  return L.dk <= 64 ? forward<64>(forward_split(L), stream) : forward<128>(forward_split(L), stream);
}

hipError_t launch_delta_step(const DeltaLaunch& L, hipStream_t stream) {
  return L.in_bf16 ? step_of<bf16>(L, stream) : step_of<float>(L, stream);
}

}  // namespace gdnq

// Gradients of the chunked delta rule (formulas in delta_common.h and below).
#include <type_traits>

#include "delta_common.h"
#include "delta_prep.h"

namespace gdnq {
namespace {

// The workspace goes on with dS' and z of every chunk and head, as the carry
// holds S and w.
__host__ __device__ inline int64_t backward_left_at(const DeltaLaunch& L, int64_t slots) {
  return delta_align(slots * L.H * DELTA_CHUNK_BYTES);
}

// ---------------------------------------------------------------- the chain of dS
//
// As the forward chain, from the last chunk to the first.
template <int DK>
__global__ __launch_bounds__(256, 1) void delta_chain_back_kernel(DeltaLaunch L, int row_groups, int64_t left_at) {
  constexpr int KB = DK / 32, TILES = DK / 16;
  __shared__ __attribute__((aligned(1024))) ChainBuffer<DK> buffers[2];
  const int h = blockIdx.x / row_groups % L.H, b = blockIdx.x / row_groups / L.H, group = blockIdx.x % row_groups;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int col = group * 64 + wave * 16 + c;
  const bool mine = col < L.dv;
  const DeltaSpan s = delta_sequence(L, b);
  const int chunks = (s.tokens + 63) / 64;
  ChainLoader<DK> loader;
  loader.init(L, L.dout, h, group, wave, lane);

  f32x4 S[TILES];  // dS^T
  const int64_t state_row = ((int64_t(b) * L.H + h) * L.dv + col) * L.dk;
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    const int at = chain_row(t, g * 4);
    S[t] = f32x4{0, 0, 0, 0};
    if (L.dh_last && mine && at < L.dk) S[t] = *reinterpret_cast<const f32x4*>(L.dh_last + state_row + at);
  }
  if (chunks > 0)
    loader.template load<true>(buffers[0], s.first + int64_t(chunks - 1) * 64, s.tokens - (chunks - 1) * 64, s.slot + chunks - 1);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  for (int done = 0; done < chunks; ++done) {
    const int chunk = chunks - 1 - done;
    const ChainBuffer<DK>& buf = buffers[done & 1];
    if (chunk > 0) loader.template load<true>(buffers[(done + 1) & 1], s.first + int64_t(chunk - 1) * 64, 64, s.slot + chunk - 1);
    bf16* left = reinterpret_cast<bf16*>(static_cast<uint8_t*>(L.workspace) + left_at +
                                         ((s.slot + chunk) * L.H + h) * delta_left_bytes(L));
    bf16x8 sh[KB], sl[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      split8(S[2 * j], S[2 * j + 1], sh[j], sl[j]);
      const int at = j * 32 + g * 8;
      if (mine && at < L.dk) {
        *reinterpret_cast<bf16x8*>(left + col * L.dk + at) = sh[j];
        *reinterpret_cast<bf16x8*>(left + (L.dv + col) * L.dk + at) = sl[j];
      }
    }
    const float* rows = reinterpret_cast<const float*>(buf.rows);
    auto row4 = [&](int which, int it) { return *reinterpret_cast<const f32x4*>(rows + which * 64 + chain_row(it, g * 4)); };
    f32x4 u[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int row = chain_row(it, c);
      u[it] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < KB; ++j) u[it] = mfma_exact_split(lds_frag(buf.k + lds_block<DK>(row, j * 4 + g)), sh[j], sl[j], u[it]);
      u[it] *= row4(ROW_TAIL, it);
    }
    // dO, and c dO in parts
    bf16x8 d[2], dh[2], dl[2], hi[2], lo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const s16x4 d0 = chain_column(buf.v, 2 * j, wave, lane), d1 = chain_column(buf.v, 2 * j + 1, wave, lane);
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      d[j] = __builtin_bit_cast(bf16x8, s16x8{d0[0], d0[1], d0[2], d0[3], d1[0], d1[1], d1[2], d1[3]});
      f32x4 a = row4(ROW_C, 2 * j), b4 = row4(ROW_C, 2 * j + 1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] *= bf16_value(d0[e]);
        b4[e] *= bf16_value(d1[e]);
      }
      split8(a, b4, dh[j], dl[j]);
    }
    // transposed triangles: tiles 0 and 1 take both halves of the tokens, 2 and 3 the second
    auto block_at = [&](int it, int j) { return buf.tri + (it < 2 ? it * 2 + j : it + 2) * 1024 + lane * 16; };
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int j = it / 2; j < 2; ++j) {
        const uint8_t* at = block_at(it, j) + TRI_BYTES;
        u[it] = mfma16(lds_frag(at), d[j], mfma16(lds_frag(at + TRI_PART), d[j], u[it]));
      }
    split8(u[0], u[1], hi[0], lo[0]);
    split8(u[2], u[3], hi[1], lo[1]);
    f32x4 z[4] = {};
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int j = it / 2; j < 2; ++j) {
        const uint8_t* at = block_at(it, j);
        z[it] = mfma_split_split(lds_frag(at), lds_frag(at + TRI_PART), hi[j], lo[j], z[it]);
      }
    bf16x8 zh[2], zl[2];
    split8(z[0], z[1], zh[0], zl[0]);
    split8(z[2], z[3], zh[1], zl[1]);
#pragma unroll
    for (int it = 0; it < 4; ++it) z[it] *= -row4(ROW_C_BETA, it);
    split8(z[0], z[1], hi[0], lo[0]);
    split8(z[2], z[3], hi[1], lo[1]);
    const float whole = rows[ROW_C * 64 + 63];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      S[t] *= whole;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = j * 32 + g * 8 + (c >> 2), block = (t >> 1) * 4 + (c & 3), half = (t & 1) * 8;
        const int a = lds_block<DK>(row, block) + half, b4 = lds_block<DK>(row + 4, block) + half;
        S[t] = mfma_exact_split(lds_transposed(buf.q + a, buf.q + b4), dh[j], dl[j], S[t]);
        S[t] = mfma_exact_split(lds_transposed(buf.k + a, buf.k + b4), hi[j], lo[j], S[t]);
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (mine) {
      bf16* zp = left + 2 * L.dv * L.dk;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<bf16x8*>(zp + col * 64 + j * 32 + g * 8) = zh[j];
        *reinterpret_cast<bf16x8*>(zp + (L.dv + col) * 64 + j * 32 + g * 8) = zl[j];
      }
    }
  }
  if (L.dh0 && mine) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int at = chain_row(t, g * 4);
      if (at < L.dk) *reinterpret_cast<f32x4*>(L.dh0 + state_row + at) = S[t];
    }
  }
}

// ---------------------------------------------------------------- the gradients of a chunk
//
// With S entering, dS' leaving, u = beta w and dx = beta z:
//   dM = dO u^T (j <= i),   dAt = -dx u^T (j < i),   both times rho below
//   dQ = c dO S + dM K
//   dK = dAt K - c dx S + dM^T Q + dAt^T K + (c_64 / c) u dS'
//   d log alpha_t = sum over i >= t > j of dM_ij q_i.k_j + dAt_ij k_i.k_j
//                 + sum over i >= t of q_i.(c dO S)_i - k_i.(c dx S)_i
//                 + sum over j < t of k_j.((c_64 / c) u dS')_j  + c_64 <S, dS'>
// A sum over what passes token t, with nothing subtracted: what lies before or
// behind it wholly is not in it.
//   One workgroup per chunk and key head, wave it the 16 tokens of tile it,
// over the key head's value heads in turn (so that their sum needs no atomics
// and no memory).  S and dS' pass through LDS 32 rows (d_v) at a time.
template <int DK>
__global__ __launch_bounds__(256, 1) void delta_gradient_kernel(DeltaLaunch L, int64_t left_at) {
  constexpr int BLOCKS = DK / 8, KB = DK / 32, TILES = DK / 16;
  constexpr int MAT = 64 * DK * 2, LOADS = 64 * BLOCKS / 256, SLAB = 32 * DK * 2, SLAB_LOADS = 4 * 32 * BLOCKS / 256;
  __shared__ __attribute__((aligned(1024))) uint8_t ks[MAT], qs[MAT], slab[4 * SLAB], wz[4 * 4096], pairs[4 * 8192];
  __shared__ float rest[64], gamma[64], tail[64], beta[64], below[4][64], row_in[64], row_out[64], pair_sum[64], dots[4];
  __shared__ int whole[64];
  const int64_t slot = blockIdx.x / L.G;
  const int kh = blockIdx.x % L.G, share = L.H / L.G;
  int64_t first;
  const int n = delta_slot_tokens(L, slot, first);
  if (n == 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int64_t krow = int64_t(L.G) * L.dk, vrow = int64_t(L.H) * L.dv;
  const uint8_t* space = static_cast<const uint8_t*>(L.workspace);
  {
    const bf16* kp = static_cast<const bf16*>(L.k) + int64_t(kh) * L.dk;
    const bf16* qp = static_cast<const bf16*>(L.q) + int64_t(kh) * L.dk;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int p = i * 256 + threadIdx.x, row = p / BLOCKS, block = p % BLOCKS, to = lds_block<DK>(row, block);
      const bool keep = row < n && block * 8 < L.dk;
      const int64_t at = (first + min(row, n - 1)) * krow + min(block * 8, L.dk - 8);
      *reinterpret_cast<u32x4*>(ks + to) = only_if(keep, *reinterpret_cast<const u32x4*>(kp + at));
      *reinterpret_cast<u32x4*>(qs + to) = only_if(keep, *reinterpret_cast<const u32x4*>(qp + at));
    }
  }
  __syncthreads();
  // q.k and k.k of the wave's rows with the tokens up to them: exact products
  f32x4 qk[4] = {}, kk[4] = {};
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    const int at = lds_block<DK>(wave * 16 + c, j * 4 + g);
    const bf16x8 qr = lds_frag(qs + at), kr = lds_frag(ks + at);
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      if (jt > wave) break;
      const bf16x8 kc = lds_frag(ks + lds_block<DK>(jt * 16 + c, j * 4 + g));
      qk[jt] = mfma16(qr, kc, qk[jt]);
      kk[jt] = mfma16(kr, kc, kk[jt]);
    }
  }
  // the first operand's row of this lane, and a row of it out of memory
  const int token = wave * 16 + c;
  const bool here = token < n;
  const int64_t at_row = (first + (here ? token : 0)) * vrow;
  const bf16* dop = static_cast<const bf16*>(L.dout) + at_row;
  bf16* dvp = static_cast<bf16*>(L.dv_out) + at_row;
  // 4 x 16 (row, column) blocks of a transposing read
  const int tr_row = g * 8 + (c >> 2), tr_half = (c & 1) * 8;

  f32x4 dq[TILES] = {}, dk[TILES] = {};
  for (int hs = 0; hs < share; ++hs) {
    const int h = kh * share + hs;
    const int64_t chunk = slot * L.H + h;
    if (threadIdx.x < 64) {
      const float* sc = reinterpret_cast<const float*>(space + chunk * DELTA_CHUNK_BYTES + DELTA_SCALARS) + lane;
      gamma[lane] = sc[ROW_C * 64];
      tail[lane] = sc[ROW_TAIL * 64];
      beta[lane] = sc[ROW_BETA * 64];
      whole[lane] = reinterpret_cast<const int*>(sc)[ROW_WHOLE * 64];
      rest[lane] = sc[ROW_REST * 64];
    }
    const bf16* states = reinterpret_cast<const bf16*>(static_cast<const uint8_t*>(L.carry) + chunk * delta_left_bytes(L));
    const bf16* dstates = reinterpret_cast<const bf16*>(space + left_at + chunk * delta_left_bytes(L));
    f32x4 ds[TILES] = {}, xs[TILES] = {}, ud[TILES] = {};  // dO S, z S, w dS'
    f32x4 dm[4] = {}, da[4] = {};
    float db = 0.0f, dot = 0.0f;
    __syncthreads();
    const float bt = beta[token];
    for (int v0 = 0; v0 < L.dv; v0 += 32) {
      // parts: S hi, S lo, dS' hi, dS' lo
#pragma unroll
      for (int i = 0; i < SLAB_LOADS; ++i) {
        const int p = i * 256 + threadIdx.x, part = p / (32 * BLOCKS), row = p / BLOCKS % 32, block = p % BLOCKS;
        const bool keep = v0 + row < L.dv && block * 8 < L.dk;
        const u32x4 x = *reinterpret_cast<const u32x4*>((part < 2 ? states : dstates) +
                                                        (int64_t(part & 1) * L.dv + min(v0 + row, L.dv - 1)) * L.dk +
                                                        min(block * 8, L.dk - 8));
        *reinterpret_cast<u32x4*>(slab + part * SLAB + lds_block<DK>(row, block)) = only_if(keep, x);
      }
      // w hi, w lo, z hi, z lo: 32 rows of 64 tokens each
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = threadIdx.x / 8, block = threadIdx.x % 8;
        const u32x4 x = *reinterpret_cast<const u32x4*>((i < 2 ? states : dstates) + 2 * int64_t(L.dv) * L.dk +
                                                        (int64_t(i & 1) * L.dv + min(v0 + row, L.dv - 1)) * 64 + block * 8);
        *reinterpret_cast<u32x4*>(wz + i * 4096 + lds_block<64>(row, block)) = only_if(v0 + row < L.dv, x);
      }
      const bool keep = here && v0 + g * 8 < L.dv;
      const int64_t at = int64_t(h) * L.dv + min(v0 + g * 8, L.dv - 8);
      const bf16x8 o8 = __builtin_bit_cast(bf16x8, only_if(keep, *reinterpret_cast<const u32x4*>(dop + at)));
      __syncthreads();
      // the wave's tokens of w and z, in parts: rows of the first operand
      auto tokens16 = [&](const uint8_t* part, int tile) {
        const int block = tile * 2 + ((c & 3) >> 1);
        return lds_transposed(part + lds_block<64>(tr_row, block) + tr_half, part + lds_block<64>(tr_row + 4, block) + tr_half);
      };
      const bf16x8 wh = tokens16(wz, wave), wl = tokens16(wz + 4096, wave);
      const bf16x8 zh = tokens16(wz + 8192, wave), zl = tokens16(wz + 12288, wave);
      bf16x8 dv8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = float(zh[e]) + float(zl[e]);
        db = fmaf(float(wh[e]) + float(wl[e]), z, db);
        dv8[e] = bf16(bt * z);
      }
      if (keep) *reinterpret_cast<bf16x8*>(dvp + at) = dv8;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const int block = t * 2 + ((c & 3) >> 1);
        const int a = lds_block<DK>(tr_row, block) + tr_half, b = lds_block<DK>(tr_row + 4, block) + tr_half;
        const bf16x8 sh = lds_transposed(slab + a, slab + b), sl = lds_transposed(slab + SLAB + a, slab + SLAB + b);
        const bf16x8 dh = lds_transposed(slab + 2 * SLAB + a, slab + 2 * SLAB + b);
        const bf16x8 dl = lds_transposed(slab + 3 * SLAB + a, slab + 3 * SLAB + b);
        ds[t] = mfma_exact_split(o8, sh, sl, ds[t]);
        xs[t] = mfma_split_split(zh, zl, sh, sl, xs[t]);
        ud[t] = mfma_split_split(wh, wl, dh, dl, ud[t]);
      }
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        if (jt > wave) break;
        const bf16x8 h8 = tokens16(wz, jt), l8 = tokens16(wz + 4096, jt);
        dm[jt] = mfma_exact_split(o8, h8, l8, dm[jt]);
        da[jt] = mfma_split_split(zh, zl, h8, l8, da[jt]);
      }
      // <S, dS'> of the slab's 32 rows
#pragma unroll
      for (int i = 0; i < 32 * BLOCKS / 256; ++i) {
        const int p = (i * 256 + threadIdx.x) * 16;
        const bf16x8 sh = lds_frag(slab + p), sl = lds_frag(slab + SLAB + p);
        const bf16x8 dh = lds_frag(slab + 2 * SLAB + p), dl = lds_frag(slab + 3 * SLAB + p);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(float(sh[e]) + float(sl[e]), float(dh[e]) + float(dl[e]), dot);
      }
      __syncthreads();
    }
    db = xor32_sum(xor16_sum(db));
    if (here && g == 0) L.dbeta[(first + token) * L.H + h] = db;
    dot = wave_allreduce_sum(dot);
    if (lane == 0) dots[wave] = dot;

    // The triangles times rho, in two parts, by columns: row j of `pairs` holds
    // the 64 tokens i.  And what passes each token (sums from the last row up).
    f32x4 passing[4] = {};
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      if (jt > (wave | 1)) break;
      const int j = jt * 16 + c;
      float m4[4], a4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = wave * 16 + g * 4 + e;
        const float rho = j <= i ? exp2_difference(rest[i], whole[i], rest[j], whole[j]) : 0.0f;
        m4[e] = rho * beta[j] * dm[jt][e];
        a4[e] = j < i ? -rho * beta[j] * beta[i] * da[jt][e] : 0.0f;
        passing[jt][e] = j <= i ? m4[e] * qk[jt][e] + a4[e] * kk[jt][e] : 0.0f;
      }
      const int to = lds_block<64>(j, wave * 2 + (g >> 1)) + (g & 1) * 8;
      bf16x4 hi, lo;
      split2(m4, hi, lo);
      *reinterpret_cast<bf16x4*>(pairs + to) = hi;
      *reinterpret_cast<bf16x4*>(pairs + 8192 + to) = lo;
      split2(a4, hi, lo);
      *reinterpret_cast<bf16x4*>(pairs + 16384 + to) = hi;
      *reinterpret_cast<bf16x4*>(pairs + 24576 + to) = lo;
      // sums over the rows from e on, then with those of the lane groups below
#pragma unroll
      for (int e = 2; e >= 0; --e) passing[jt][e] += passing[jt][e + 1];
      const float own = passing[jt][0];
      const float up1 = __shfl_down(own, 16), up2 = __shfl_down(own, 32), up3 = __shfl_down(own, 48);
      const float behind = (g < 3 ? up1 : 0.0f) + (g < 2 ? up2 : 0.0f) + (g < 1 ? up3 : 0.0f);
#pragma unroll
      for (int e = 0; e < 4; ++e) passing[jt][e] += behind;
      if (g == 0) below[wave][j] = passing[jt][0];
    }
    __syncthreads();
    {
      f32x4 sum = {0, 0, 0, 0};
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        if (jt > wave) break;
        float later = 0.0f;
        for (int it = wave + 1; it < 4; ++it) later += below[it][jt * 16 + c];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (jt * 16 + c < wave * 16 + g * 4 + e) sum[e] += passing[jt][e] + later;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum[e] = group_sum<16>(sum[e]);
        if (c == 0) pair_sum[wave * 16 + g * 4 + e] = sum[e];
      }
    }
    // dM K, dAt K (rows i), dM^T Q, dAt^T K (rows j)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (kb <= wave / 2) {  // j up to the wave's rows
        const int block = wave * 2 + ((c & 3) >> 1);
        const int a = lds_block<64>(kb * 32 + tr_row, block) + tr_half, b = lds_block<64>(kb * 32 + tr_row + 4, block) + tr_half;
        const bf16x8 mh = lds_transposed(pairs + a, pairs + b), ml = lds_transposed(pairs + 8192 + a, pairs + 8192 + b);
        const bf16x8 ah = lds_transposed(pairs + 16384 + a, pairs + 16384 + b);
        const bf16x8 al = lds_transposed(pairs + 24576 + a, pairs + 24576 + b);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          const int block = t * 2 + ((c & 3) >> 1);
          const int ka = lds_block<DK>(kb * 32 + tr_row, block) + tr_half, kb4 = lds_block<DK>(kb * 32 + tr_row + 4, block) + tr_half;
          const bf16x8 k8 = lds_transposed(ks + ka, ks + kb4);
          dq[t] = mfma16(mh, k8, mfma16(ml, k8, dq[t]));
          dk[t] = mfma16(ah, k8, mfma16(al, k8, dk[t]));
        }
      }
      if (kb >= wave / 2) {  // i from the wave's rows on
        const int at = lds_block<64>(wave * 16 + c, kb * 4 + g);
        const bf16x8 mh = lds_frag(pairs + at), ml = lds_frag(pairs + 8192 + at);
        const bf16x8 ah = lds_frag(pairs + 16384 + at), al = lds_frag(pairs + 24576 + at);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          const int block = t * 2 + ((c & 3) >> 1);
          const int ka = lds_block<DK>(kb * 32 + tr_row, block) + tr_half, kb4 = lds_block<DK>(kb * 32 + tr_row + 4, block) + tr_half;
          const bf16x8 q8 = lds_transposed(qs + ka, qs + kb4), k8 = lds_transposed(ks + ka, ks + kb4);
          dk[t] = mfma16(mh, q8, mfma16(ml, q8, dk[t]));
          dk[t] = mfma16(ah, k8, mfma16(al, k8, dk[t]));
        }
      }
    }
    // what the state gives, and its share of the decays' gradient
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = wave * 16 + g * 4 + e;
      const float gm = gamma[row], gb = gm * beta[row], tb = tail[row] * beta[row];
      float in = 0.0f, out = 0.0f;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const int at = lds_block<DK>(row, t * 2 + (c >> 3)) + (c & 7) * 2;
        const float q = float(*reinterpret_cast<const bf16*>(qs + at)), k = float(*reinterpret_cast<const bf16*>(ks + at));
        const float a = gm * ds[t][e], x = gb * xs[t][e], u = tb * ud[t][e];
        in = fmaf(q, a, fmaf(-k, x, in));
        out = fmaf(k, u, out);
        dq[t][e] += a;
        dk[t][e] += u - x;
      }
      in = group_sum<16>(in);
      out = group_sum<16>(out);
      if (c == 0) row_in[row] = in, row_out[row] = out;
    }
    __syncthreads();
    if (wave == 0) {
      // sums over i >= t, and over j < t (not of all up to t less the token's own:
      // its own is far larger where the token forgets much)
      float in = row_in[63 - lane], out = lane ? row_out[lane - 1] : 0.0f;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const float a = __shfl_up(in, d), b = __shfl_up(out, d);
        if (lane >= d) in += a, out += b;
      }
      in = __shfl(in, 63 - lane);
      float da_t = pair_sum[lane] + in + out + gamma[63] * (dots[0] + dots[1] + dots[2] + dots[3]);
      if (lane < n) {
        const int64_t at = (first + lane) * L.H + h;
        if (!L.log_decay) {
          const float a = L.alpha[at];
          da_t /= fmaxf(a, 5.42101086e-20f);  // the least decay, 2^-64
        }
        L.dalpha[at] = da_t;
      }
    }
    __syncthreads();
  }
  bf16* dqp = static_cast<bf16*>(L.dq) + int64_t(kh) * L.dk;
  bf16* dkp = static_cast<bf16*>(L.dk_out) + int64_t(kh) * L.dk;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int row = wave * 16 + g * 4 + e;
    if (row >= n) continue;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      if (t * 16 + c >= L.dk) continue;
      store_f32(dqp + (first + row) * krow + t * 16 + c, dq[t][e]);
      store_f32(dkp + (first + row) * krow + t * 16 + c, dk[t][e]);
    }
  }
}

template <int DK>
hipError_t backward(const DeltaLaunch& L, hipStream_t stream) {
  const int64_t slots = delta_slots(L);
  const int64_t left_at = backward_left_at(L, slots);
  if (slots > 0) {
    delta_prep_kernel<DK, true><<<uint32_t(slots * L.H), 256, 0, stream>>>(L);
    if (hipError_t e = hipGetLastError()) return e;
  }
  const int groups = (L.dv + 63) / 64;
  delta_chain_back_kernel<DK><<<uint32_t(groups) * uint32_t(L.H) * uint32_t(L.B), 256, 0, stream>>>(L, groups, left_at);
  if (hipError_t e = hipGetLastError()) return e;
  if (slots > 0) delta_gradient_kernel<DK><<<uint32_t(slots * L.G), 256, 0, stream>>>(L, left_at);
  return hipGetLastError();
}

}  // namespace

size_t delta_backward_workspace_bytes(const DeltaLaunch& L) {
  const int64_t slots = delta_slots(L);
  return size_t(backward_left_at(L, slots) + slots * L.H * delta_left_bytes(L));
}

hipError_t launch_delta_backward(const DeltaLaunch& L, hipStream_t stream) {
  return L.dk <= 64 ? backward<64>(L, stream) : backward<128>(L, stream);
}

}  // namespace gdnq

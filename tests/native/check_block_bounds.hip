// Host-side check of the block-scaled kernels' addressing: runs, on the CPU,
// the code with which the GPU kernels address their loads (BlockGemm::lanes /
// live / access, BlockRowsN::dma_* / read_*, BlockGrad::lanes) for every tile,
// stage, wave and lane of many problems, and checks that
//   1. every enabled access starts inside the valid rows and columns of its
//      matrix, at an offset that a buffer reaches (below 2^31);
//   2. every valid chunk of a stage arrives exactly once, at the LDS place where
//      the operand reads look for it;
//   3. every row's (or block of columns') scale arrives once;
//   4. a stage past a slice's end loads nothing.
// Prints "ALL OK" and exits 0, or prints the first violations and exits 1.
// Build: hipcc --cuda-host-only -std=c++17 -I include -I <csrc> check_block_bounds.hip
#include <algorithm>
#include <cstdio>
#include <utility>
#include <vector>

#include "bst_block_gemm.hpp"
#include "bst_block_grad.hpp"
#include "bst_block_rows.hpp"

using namespace bst;

static int g_fail = 0;
static long long g_checked = 0;

#define REQUIRE(cond, ...)                               \
  do {                                                   \
    if (!(cond)) {                                       \
      if (g_fail < 10) {                                 \
        printf("VIOLATION %s:%d: ", __FILE__, __LINE__); \
        printf(__VA_ARGS__);                             \
        printf("\n");                                    \
      }                                                  \
      ++g_fail;                                          \
    }                                                    \
  } while (0)

struct Size {
  int64_t M, N, K, padA, padB, padS;
};

template <typename F, size_t... X>
static void each(F f, std::index_sequence<X...>) {
  (f(std::integral_constant<int, (int)X>{}), ...);
}

static int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

template <int BM, int BN, int WM, int WN, int ST, bool TB>
void gemm(const Size& z) {
  using KN = BlockGemm<BM, BN, WM, WN, ST, TB, MODE_F32, false>;
  const int64_t lda = up(z.K, 16) + z.padA, ldb = up(TB ? z.K : z.N, 16) + z.padB;
  const int64_t kb = up(z.K, 128) / 128, nb = up(z.N, 128) / 128;
  const int64_t ldsa = kb + z.padS, ldsb = (TB ? kb : nb) + z.padS;
  const uint32_t nk = (uint32_t)kb;
  for (int64_t m0 = 0; m0 < z.M; m0 += BM)
    for (int64_t n0 = 0; n0 < z.N; n0 += BN) {
      const uint32_t rows = (uint32_t)std::min<int64_t>(BM, z.M - m0);
      const uint32_t cols = (uint32_t)std::min<int64_t>(BN, z.N - n0);
      for (uint32_t kt = 0; kt <= nk; ++kt) {
        std::vector<int> seen((KN::A_BYTES + KN::B_BYTES) / 16), sa(BM), sb((BN + 127) / 128);
        const int64_t left = z.K - (int64_t)kt * 128;  // K rows from this stage on
        for (uint32_t wave = 0; wave < (uint32_t)KN::NW; ++wave) {
          const bool for_a = wave < (uint32_t)KN::SA_N;
          const typename KN::Tile tile{(uint32_t)lda, (uint32_t)ldb, (uint32_t)z.K, rows, cols,
                                       (uint32_t)((for_a ? ldsa : TB ? ldsb : 1) * 4),
                                       (uint32_t)(nb - n0 / 128)};
          for (uint32_t lane = 0; lane < 64; ++lane) {
            const typename KN::Lanes ln = KN::lanes(tile, wave, lane);
            const uint32_t bits = KN::live(ln, kt, nk, (uint32_t)z.K);
            each([&](auto xx) {
              constexpr int X = decltype(xx)::value;
              const typename KN::Access c = KN::template access<X>(
                  wave, (uint32_t)lda, (uint32_t)ldb, ln, bits, ln.a_ch, ln.b_ch);
              ++g_checked;
              const uint32_t at = c.lds + lane * 16;
              REQUIRE(at + 16 <= (uint32_t)(KN::A_BYTES + KN::B_BYTES), "LDS place %u", at);
              if (c.voff == kOob) return;
              REQUIRE(kt < nk, "a load past the last stage");
              const int64_t off = (int64_t)c.voff + c.soff;
              REQUIRE(off + 16 <= (int64_t)kOob, "offset %lld", (long long)off);
              const bool a = X < KN::A_IPW;
              const int64_t ld = a ? lda : ldb, row = off / ld, byte = off % ld;
              uint32_t want;
              if (a || TB) {  // rows of 128 bytes, chunks XORed by the row
                REQUIRE(row < (a ? rows : cols), "row %lld", (long long)row);
                REQUIRE(byte % 16 == 0 && byte < std::min<int64_t>(128, left), "byte %lld of K",
                        (long long)byte);
                want = (uint32_t)row * 128 + (((uint32_t)(byte / 16) ^ swz((uint32_t)row)) << 4);
              } else {  // K rows of BN bytes
                REQUIRE(row < std::min<int64_t>(128, left), "K row %lld", (long long)row);
                REQUIRE(byte % 16 == 0 && byte < cols, "column %lld", (long long)byte);
                want = (uint32_t)row * BN + (((uint32_t)(byte / 16) ^ KN::swz_b((uint32_t)row)) << 4);
              }
              REQUIRE(at == (a ? 0 : (uint32_t)KN::A_BYTES) + want, "LDS place %u, expected %u", at, want);
              ++seen[std::min<uint32_t>(at / 16, (uint32_t)seen.size() - 1)];
            }, std::make_index_sequence<KN::ND>());
            if (kt < nk && ln.s_off != kOob) {
              const uint32_t i = ln.s_off / tile.s_pitch;
              REQUIRE(ln.s_off % tile.s_pitch == 0 && (for_a || wave == (uint32_t)KN::SA_N), "scale offset");
              REQUIRE(i < (for_a ? rows : up(cols, 128) / 128), "scale of row or block %u", i);
              if (i < (for_a ? sa : sb).size()) ++(for_a ? sa : sb)[i];
            }
          }
        }
        if (kt == nk) continue;
        const int64_t ch = up(std::min<int64_t>(128, left), 16) / 16;
        const int64_t expect = rows * ch + (TB ? cols * ch : std::min<int64_t>(128, left) * (up(cols, 16) / 16));
        int64_t n = 0;
        for (int s : seen) {
          REQUIRE(s <= 1, "a chunk arrives %d times", s);
          n += s;
        }
        REQUIRE(n == expect, "%lld chunks of %lld", (long long)n, (long long)expect);
        for (uint32_t r = 0; r < rows; ++r) REQUIRE(sa[r] == 1, "row %u's scale arrives %d times", r, sa[r]);
        for (uint32_t b = 0; b < up(cols, 128) / 128; ++b) REQUIRE(sb[b] == 1, "block %u's scale", b);
      }
    }
}

void rows_n(const Size& z) {
  using KN = BlockRowsN<1, false>;
  const int64_t ldb = up(z.N, 16) + z.padB;
  for (int64_t n0 = 0; n0 < z.N; n0 += KN::BN)
    for (int64_t k0 = 0; k0 < z.K; k0 += 128) {
      const uint32_t cols = (uint32_t)std::min<int64_t>(KN::BN, z.N - n0), left = (uint32_t)(z.K - k0);
      std::vector<int> seen(KN::BUF / 16), read(KN::BUF / 8);
      for (uint32_t lane = 0; lane < 64; ++lane) {
        const KN::Lane l = KN::dma_lane(lane, (uint32_t)ldb, cols);
        for (int x = 0; x < KN::DMAS; ++x) {
          ++g_checked;
          const uint32_t v = KN::dma_voff(l, x, left), at = x * 1024 + lane * 16;
          if (v == kOob) continue;
          const int64_t off = (int64_t)v + KN::dma_soff(x, (uint32_t)ldb), k = off / ldb, c = off % ldb;
          REQUIRE(off + 16 <= (int64_t)kOob, "offset %lld", (long long)off);
          REQUIRE(k < std::min<uint32_t>(128, left) && c % 16 == 0 && c < cols, "K row %lld column %lld",
                  (long long)k, (long long)c);
          REQUIRE(at == k * KN::BN + ((c / 16 ^ KN::swz_n((uint32_t)k)) << 4), "LDS place %u", at);
          ++seen[at / 16];
        }
        for (int kk = 0; kk < 2; ++kk)
          for (int t = 0; t < 4; ++t) {
            const uint32_t at = KN::read_off(lane) + KN::read_step(kk, t);
            REQUIRE(at % 8 == 0 && at + 8 <= (uint32_t)KN::BUF, "read at %u", at);
            if (at / 8 < read.size()) ++read[at / 8];
          }
      }
      int64_t n = 0;
      for (int s : seen) n += s;
      REQUIRE(n == (int64_t)std::min<uint32_t>(128, left) * (up(cols, 16) / 16) &&
                  *std::max_element(seen.begin(), seen.end()) <= 1, "%lld chunks", (long long)n);
      REQUIRE(*std::min_element(read.begin(), read.end()) == 1 &&
                  *std::max_element(read.begin(), read.end()) == 1, "a patch is read once");
    }
}

template <int BK, int BN, int WM, int WN, int DY>
void grad(const Size& z) {
  using KN = BlockGrad<BK, BN, WM, WN, DY>;
  constexpr uint32_t ES = DY == DY_F32 ? 4 : 2, XR = KN::NT / KN::XCH, YR = KN::NT / KN::YCH;
  const int64_t ldq = up(z.K, 16) + z.padA, ldy = (up(z.N * ES, 16) + z.padB) / ES * ES;
  const int64_t lds = up(z.K, 128) / 128 + z.padS;
  for (int64_t k0 = 0; k0 < z.K; k0 += BK)
    for (int64_t n0 = 0; n0 < z.N; n0 += BN)
      for (int64_t r0 = 0; r0 < z.M; r0 += KN::D) {
        typename KN::Src c{};
        c.ldq = ldq;
        c.lds = lds;
        c.ldy = ldy;
        c.kcols = (uint32_t)std::min<int64_t>(BK, z.K - k0);
        c.ncols = (uint32_t)std::min<int64_t>(BN, z.N - n0);
        c.rows = (uint32_t)z.M;
        const uint32_t left = (uint32_t)(z.M - r0);
        int64_t nx = 0, ny = 0;
        for (uint32_t tid = 0; tid < (uint32_t)KN::NT; ++tid) {
          const typename KN::Lanes l = KN::lanes(c, tid);
          for (uint32_t i = 0; i < (uint32_t)KN::XL; ++i) {
            ++g_checked;
            if (!(i * XR + tid / KN::XCH < left) || l.x == kOob) continue;
            const int64_t off = (int64_t)l.x + i * XR * (uint32_t)ldq, so = (int64_t)l.e + i * XR * (uint32_t)lds;
            REQUIRE(off + 16 <= (int64_t)kOob && so < (int64_t)kOob, "offsets %lld %lld", (long long)off, (long long)so);
            REQUIRE(off / ldq < std::min<uint32_t>(left, KN::D) && off % ldq < c.kcols && off % ldq % 16 == 0,
                    "codes at %lld", (long long)off);
            REQUIRE(so / lds == off / ldq && so % lds == off % ldq / 128, "scale at %lld", (long long)so);
            ++nx;
          }
          for (uint32_t i = 0; i < (uint32_t)KN::YL; ++i)
            for (int w = 0; w < (DY == DY_F32 ? 2 : 1); ++w) {
              if (!(i * YR + tid / KN::YCH < left) || l.y[w] == kOob) continue;
              const int64_t off = (int64_t)l.y[w] + i * YR * (uint32_t)ldy;
              REQUIRE(off + 16 <= (int64_t)kOob, "offset %lld", (long long)off);
              REQUIRE(off / ldy < std::min<uint32_t>(left, KN::D) && off % ldy < (int64_t)c.ncols * ES &&
                          off % ldy % 16 == 0, "gradients at %lld", (long long)off);
              ++ny;
            }
        }
        const int64_t live = std::min<uint32_t>(left, KN::D);
        REQUIRE(nx == live * (up(c.kcols, 16) / 16) && ny == live * (up((int64_t)c.ncols * ES, 16) / 16),
                "%lld and %lld loads", (long long)nx, (long long)ny);
      }
}

int main() {
  const std::vector<Size> sizes = {
      {1, 1, 1, 0, 0, 0},        {1, 16, 128, 16, 0, 1},   {33, 257, 129, 0, 16, 0},
      {64, 300, 1000, 16, 48, 2}, {129, 136, 256, 0, 0, 0}, {300, 520, 392, 32, 16, 3},
      {257, 129, 383, 0, 0, 1},  {7, 72, 2055, 16, 16, 0}, {65, 640, 15, 0, 0, 0}};
  for (const Size& z : sizes) {
    gemm<32, 128, 1, 4, 4, true>(z);
    gemm<32, 128, 1, 4, 4, false>(z);
    gemm<64, 128, 2, 4, 4, true>(z);
    gemm<64, 128, 2, 4, 4, false>(z);
    gemm<128, 128, 2, 4, 4, true>(z);
    gemm<128, 128, 2, 4, 4, false>(z);
    gemm<256, 256, 2, 4, 2, true>(z);
    gemm<256, 256, 2, 4, 2, false>(z);
    rows_n(z);
    grad<128, 128, 2, 2, DY_BF16>(z);
    grad<256, 256, 2, 4, DY_BF16>(z);
    grad<128, 128, 2, 2, DY_F16>(z);
    grad<256, 256, 2, 4, DY_F16>(z);
    grad<128, 128, 2, 2, DY_F32>(z);
    grad<256, 256, 2, 4, DY_F32>(z);
  }
  // the longest pitches that the host takes: 256 (K x N weights: 128) rows of
  // codes, 256 of scales and 64 of a gradient below 2 GiB
  const int64_t p256 = (1LL << 23) - 1024, p128 = (1LL << 24) - 2048, p64 = (1LL << 25) - 4096;
  gemm<256, 256, 2, 4, 2, true>({256, 256, 272, p256, p256, (1LL << 21) - 16});
  gemm<256, 256, 2, 4, 2, false>({256, 256, 272, p256, p128, (1LL << 21) - 16});
  gemm<128, 128, 2, 4, 4, false>({128, 128, 272, p256, p128, 0});
  rows_n({1, 64, 272, 0, p128, 0});
  grad<256, 256, 2, 4, DY_BF16>({64, 256, 272, p64, p64, (1LL << 23) - 16});
  grad<128, 128, 2, 2, DY_F32>({64, 128, 272, p64, p64, 0});
  if (g_fail) {
    printf("%d violations\n", g_fail);
    return 1;
  }
  printf("ALL OK (%lld accesses)\n", g_checked);
  return 0;
}

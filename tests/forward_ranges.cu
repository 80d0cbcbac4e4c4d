// Which K/V tiles a unit of the forward kernel loads and which of them its query tiles visit, on the host: the kernel's
// own functions against the visible keys by their definition.  Prints the first failure and returns 1.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "attn_fwd_ws.cuh"

using namespace thd;

static bool sees(const SeqInfo& s, const AttnParams& p, int code, long long i, long long j) {
  const long long shift = code == kMaskCausalBottomRight ? s.kv_len - s.q_len : 0;
  if (j < 0 || j >= s.kv_len || (code != kMaskPadding && j > i + shift)) return false;
  const bool near = (p.win_left < 0 || j >= i + shift - p.win_left) && (p.win_right < 0 || j <= i + shift + p.win_right);
  return near || j < p.sinks;
}

// A tile's keys that some row sees: [first keys' end) and a run behind it, as visited tiles of 128.
template <int kWin>
static const char* check(const AttnParams& p, int code, int q_len, int kv_len, bool head_pair) {
  SeqInfo s{};
  s.q_len = q_len;
  s.kv_len = kv_len;
  set_visibility(s, code, p);
  const int rows_blk = head_pair ? kTileM : 2 * kTileM;
  for (int qb = 0; qb * rows_blk < q_len; ++qb) {
    WsUnit u{};
    for (int t = 0; t < 2; ++t) {
      u.t[t].seq = s;
      u.t[t].q0 = head_pair ? qb * kTileM : qb * rows_blk + t * kTileM;
      ws_tile_range<kWin>(u.t[t], p);
    }
    ws_share_tiles<kWin>(u);
    const int tiles = (kv_len + kBlockN - 1) / kBlockN;
    std::vector<int> loaded(tiles + 1, 0);
    int last = -1;
    for (int i = 0; i < u.n_all; ++i) {
      const int j = kWin == kWinSinks ? ws_ring_tile(i, u.nsb, u.jb) : u.jb + i;
      if (j <= last || j >= tiles) return "the ring's tiles do not ascend inside the sequence";
      last = j;
      loaded[j] = 1;
      bool any = false;
      for (int t = 0; t < 2; ++t) any = any || ws_visits<kWin>(u.t[t].ns, u.t[t].j0, u.t[t].n, j);
      if (!any) return "a tile is loaded that no query tile visits";
    }
    for (int t = 0; t < 2; ++t) {
      const WsTile& x = u.t[t];
      const int ns = kWin == kWinSinks ? x.ns : 0, j0 = kWin ? x.j0 : 0;
      int at = 0;   // the softmax warps' count of the tile's visits
      for (int j = 0; j < tiles; ++j) {
        const bool visited = loaded[j] && ws_visits<kWin>(x.ns, x.j0, x.n, j);
        bool needed = false;   // rows are 128, so the corners of the visible set are rows and columns at its ends
        for (int r = 0; r < kTileM && x.q0 + r < q_len && !needed; ++r)
          for (int c = 0; c < kBlockN && !needed; ++c) needed = sees(s, p, code, x.q0 + r, (long long)j * kBlockN + c);
        if (needed && !visited) return "a tile with a visible key is not visited";
        if (visited) {
          if ((kWin == kWinSinks ? ws_ring_tile(at, ns, j0) : j0 + at) != j) return "softmax and products count differently";
          if ((at == 0) != !(j > (ns > 0 ? 0 : j0))) return "the first product does not start the sum";
          ++at;
        }
      }
      if (at != (x.n > 0 ? ns + x.n - j0 : 0)) return "the count of a tile's visits is wrong";
    }
  }
  return nullptr;
}

int main() {
  const int kv[] = {0, 1, 100, 128, 129, 255, 256, 384, 500, 640, 1024};
  const int q[] = {129, 250, 256, 257, 384, 600, 900, 1400};
  const int bounds[][2] = {{-1, -1}, {0, -1}, {0, 0}, {5, 0}, {127, -1}, {128, 37}, {300, 7}, {-1, 40}, {1000, 0}};
  const int sinks[] = {0, 1, 4, 128, 130, 300, 2000};
  for (int code = 0; code <= 2; ++code)
    for (int n : q)
      for (int m : kv)
        for (const auto& w : bounds)
          for (int f : sinks)
            for (int pair = 0; pair < 2; ++pair) {
              AttnParams p{};
              p.win_left = w[0];
              p.win_right = w[1];
              const bool win = w[0] >= 0 || w[1] >= 0;
              p.sinks = win ? f : 0;
              const char* e = !win ? check<0>(p, code, n, m, pair) :
                              p.sinks ? check<kWinSinks>(p, code, n, m, pair) : check<1>(p, code, n, m, pair);
              if (e) {
                std::printf("%s: mask type %d, %d queries, %d keys, window (%d, %d), %d first keys, heads %s\n", e, code, n,
                            m, w[0], w[1], f, pair ? "in pairs" : "apart");
                return 1;
              }
            }
  return 0;
}

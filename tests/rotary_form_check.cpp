// Steps dl::Form and dl::HeadWalk (csrc/dl_rotary_form.h) over heads of up to
// 2^31 - 1 elements and tokens of up to 2^31 - 1 heads: every element and every
// head is taken exactly once, and none outside.
#include <cstdio>
#include <vector>

#include "dl_rotary_form.h"

namespace {

// Elements that unit u of a head takes, in order; false where one lies outside the head.
template <int N, bool I>
bool unit(int u, int head_dim, int pairs, int64_t& covered) {
    using F = dl::Form<N, I>;
    const int turned = F::turned(pairs);
    const bool turns = u < turned;
    const int64_t low = F::first(u, turned), apart = turns && !I ? pairs : N;
    if (low < 0 || low + N > head_dim) return false;
    covered += N;
    if (F::two(turns, static_cast<int>(low), head_dim)) {
        if (low + apart + N > head_dim) return false;
        covered += N;
    } else if (F::kTwo && low + 2 * N <= head_dim) {
        return false;  // room for a second pack that nobody takes
    }
    return true;
}

// All units of small heads; of the widest the last ones, the others being full.
template <int N, bool I>
int form(int head_dim, int pairs) {
    using F = dl::Form<N, I>;
    if (2 * pairs > head_dim || !F::fits(head_dim, pairs)) return 0;
    const int units = F::units(head_dim, pairs), first = units > 4096 ? units - 2048 : 0;
    int64_t covered = int64_t(first) * F::kSize;
    for (int u = first; u < units; ++u)
        if (!unit<N, I>(u, head_dim, pairs, covered)) return 1;
    // what is left is less than a pack, copied element by element
    return covered + F::rest(head_dim, pairs) % N == head_dim ? 0 : 2;
}

template <int N, bool I>
int forms() {
    std::vector<int> widths;
    for (int w = 2; w < 300; ++w) widths.push_back(w);
    for (int w = 0; w < 70; ++w) widths.push_back(INT32_MAX - w);
    for (int w : widths)
        for (int pairs : {1, 2, 3, 4, 5, 8, 9, 16, 24, 31, 32, 64, 100, 128, 149, 4096})
            if (const int bad = form<N, I>(w, pairs)) {
                std::printf("packs of %d, interleaved %d: head of %d, %d pairs: %d\n", N, I, w, pairs, bad);
                return 1;
            }
    return 0;
}

template <int ROWS>
int heads(int lanes, int n) {
    // the threads' walks from their own heads: all for few heads, else some
    int64_t taken = 0, want = 0;
    for (int head = 0; head < lanes; n > 1000000 ? head += lanes / 2 + 1 : ++head) {
        if (head < n) want += (int64_t(n) - 1 - head) / lanes + 1;
        int64_t next = head, steps = 0;
        for (dl::HeadWalk<ROWS> h(head, lanes, n); h.more(); h.next()) {
            if (++steps > int64_t(n) / (int64_t(ROWS) * lanes) + 1) return 1;  // goes on behind the last
            for (int r = 0; r < ROWS; ++r, next += lanes) {
                if (h.has(r) != (next < n)) return 2;
                if (!h.has(r)) continue;
                if (int64_t(h.row(r)) != next) return 3;
                ++taken;
            }
        }
    }
    return taken == want ? 0 : 4;
}

}  // namespace

int main() {
    if (forms<1, false>() || forms<2, false>() || forms<4, false>() || forms<8, false>() || forms<1, true>() ||
        forms<2, true>() || forms<4, true>() || forms<8, true>())
        return 1;
    for (int lanes : {1, 2, 8, 64, 256}) {
        std::vector<int> counts = {1, 2, 3, 5, 36, 300, 4099};
        if (lanes >= 64)
            for (int under : {0, 1, 2, 255, 256, 1022, 1023, 1024, 1025}) counts.push_back(INT32_MAX - under);
        for (int n : counts)
            if (const int bad = heads<4>(lanes, n)) {
                std::printf("%d heads, %d lanes: %d\n", n, lanes, bad);
                return 1;
            }
    }
    std::puts("ok");
}

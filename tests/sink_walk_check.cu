// Walks every unit of the bf16 sink-window gradient on the host and counts how often each
// (query, key) pair is summed into dq and into dk, dv. One case per input line:
//   B Hq Hkv N w n_sink d length_0 .. length_(B-1)
// Prints a line per case: "ok", or the first pair that is not summed exactly as often as it
// is visible.
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "sink_walk.cuh"

using namespace based;

struct Params {
    const int64_t* lengths;
    SinkSplit sp;
    FastDiv by_bhq, by_bhkv, by_hq, by_hkv, by_group;
    int Hq, N, w, n_sink, nt, units;
};

// Counts of one query head's pairs, for dq and for dk, dv.
using Counts = std::vector<unsigned char>;

template <int W>
std::string check(Params p, int B, int Hkv) {
    const size_t NN = (size_t)p.N * p.N;
    std::vector<Counts> dq(B * p.Hq, Counts(NN)), kv(B * p.Hq, Counts(NN));
    p.units = B * p.Hq * p.nt;
    for (int u = 0; u < p.units; ++u) {
        DqWalk<W> wk;
        for (wk.start(p, u);; wk.next()) {
            if (wk.ring_head() != wk.h / (p.Hq / Hkv)) return "dq: key/value head";
            for (int r = 0; r < kOwnRows && !wk.scan; ++r) {
                const int i = wk.own + r;
                if (i >= wk.len) break;
                for (int c = 0; c < W; ++c) {
                    const int j = wk.ring_row() + c;
                    const bool in = wk.sink() ? j < p.n_sink : j <= i && (j > i - p.w || j < p.n_sink);
                    if (in) ++dq[wk.b * p.Hq + wk.h][(size_t)i * p.N + j];
                }
            }
            if (wk.last()) break;
        }
    }
    p.units = B * Hkv * p.sp.units();
    for (int u = 0; u < p.units; ++u) {
        KvWalk<W> wk;
        int steps = 0;
        for (wk.start(p, u);; wk.next()) {
            if (++steps > 100000 || wk.ring_row() >= p.N || wk.h / (p.Hq / Hkv) != wk.hk) return "dk, dv: a step out of range";
            for (int r = 0; r < kOwnRows; ++r) {
                const int j = wk.own + r;
                if (j >= wk.len) break;                      // rows that are written as zeros
                const QueryRange q(wk.chunk >= 0, j, wk.len, p.w, p.n_sink);
                for (int i = std::max(wk.ring_row(), q.from); i < std::min(wk.ring_row() + W, q.end); ++i)
                    ++kv[wk.b * p.Hq + wk.h][(size_t)i * p.N + j];
            }
            if (wk.last()) break;
        }
    }
    for (int b = 0; b < B; ++b)
        for (int h = 0; h < p.Hq; ++h)
            for (int i = 0; i < p.N; ++i)
                for (int j = 0; j < p.N; ++j) {
                    const int want = i < clamped_len(p.lengths, b, p.N) && j <= i && (j > i - p.w || j < p.n_sink);
                    const size_t at = (size_t)i * p.N + j;
                    const int a = dq[b * p.Hq + h][at], c = kv[b * p.Hq + h][at];
                    if (a != want || c != want) {
                        std::ostringstream o;
                        o << "sequence " << b << " head " << h << " query " << i << " key " << j << ": dq " << a << ", dk and dv "
                          << c << ", visible " << want;
                        return o.str();
                    }
                }
    return "ok";
}

int main() {
    for (std::string line; std::getline(std::cin, line);) {
        std::istringstream in(line);
        int B, Hq, Hkv, N, w, s, d;
        in >> B >> Hq >> Hkv >> N >> w >> s >> d;
        std::vector<int64_t> lengths(B);
        for (auto& n : lengths) in >> n;
        Params p{lengths.data(), sink_split(Hq, Hkv, N, w, s, kOwnRows, d), FastDiv(B * Hq), FastDiv(B * Hkv), FastDiv(Hq),
                 FastDiv(Hkv), FastDiv(Hq / Hkv), Hq, N, w, s, (N + kOwnRows - 1) / kOwnRows, 0};
        std::puts((d == 64 ? check<64>(p, B, Hkv) : check<128>(p, B, Hkv)).c_str());
    }
}

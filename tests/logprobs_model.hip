// A host model of how the waves of a workgroup gather the top alternatives
// (csrc/logprobs.hip), with the kernel's own keys, gate and buffer size.  The
// waves' steps run in any order, and a wave reads a bound that any step before
// has published, not only the last: what the GPU's timing may do.
#include <algorithm>
#include <cmath>
#include <random>
#include <vector>

#include "logprobs_keys.h"

using namespace bqm;

namespace {

constexpr int kWaves = 4, kLanes = 64, kWaveStep = kLanes * kLpVals, kStep = kWaves * kWaveStep;
constexpr float kLowest = -3.402823466e+38f;

struct Wave {
    u64 bound = 0;
    int passed = 0, read = 0;    // read: the published bound it has seen last
    float most[kLanes];
    std::vector<u64> list, waiting;
    Wave() { std::fill(most, most + kLanes, -INFINITY); }
};

struct Model {
    const float *l;
    int n, skip, vec, top, most_waiting = 0;
    Wave w[kWaves];
    std::vector<u64> published{0};

    // lane's logit e of a step, as the kernel's 16-byte loads spread them
    int column(int st, int wave, int lane, int e) const {
        return st * kStep + wave * kWaveStep + (e / vec) * kLanes * vec + lane * vec + e % vec - skip;
    }
    bool inside(int c) const { return c >= 0 && c < n; }

    static void sort_list(std::vector<u64> &v) {
        std::sort(v.begin(), v.end(), std::greater<u64>());
        if (v.size() > kLanes) v.resize(kLanes);
    }

    bool step(int wave, int st, u64 others) {
        Wave &q = w[wave];
        float v[kLanes][kLpVals], big[kLanes];
        u64 key[kLanes][kLpVals], best[kLanes];
        for (int lane = 0; lane < kLanes; lane++) {
            big[lane] = NAN;
            best[lane] = 0;
            for (int e = 0; e < kLpVals; e++) {
                const int c = column(st, wave, lane, e);
                v[lane][e] = inside(c) ? l[c] : -INFINITY;
                key[lane][e] = inside(c) ? key_of(v[lane][e], c) : 0;
                big[lane] = fmaxf(big[lane], v[lane][e]);
                best[lane] = std::max(best[lane], key[lane][e]);
            }
        }
        q.bound = std::max(q.bound, others);
        const u64 before = q.bound;
        const LpGate gate(before, st * kStep + wave * kWaveStep - skip);
        int lanes = 0;
        for (int lane = 0; lane < kLanes; lane++) {
            lanes += gate.admits(big[lane]);
            q.most[lane] = fmaxf(q.most[lane], big[lane]);
        }
        if (lanes == 0) return true;
        q.passed += lanes;
        if (gate.open || lanes >= top || q.passed >= 8 + top / 2) {
            q.passed = 0;
            float sorted[kLanes];
            std::copy(q.most, q.most + kLanes, sorted);
            std::sort(sorted, sorted + kLanes, std::greater<float>());
            const float kth = sorted[top - 1];
            const int ties = (int)std::count(q.most, q.most + kLanes, kth);
            if (kth >= kLowest && ties <= kLpTies) {
                q.bound = std::max(q.bound, ((u64)order_of(kth) << 32) - 1);
            } else if (gate.open || lanes >= top) {
                int above = 0;
                for (int lane = 0; lane < kLanes; lane++) above += best[lane] > q.bound;
                if (above >= top) {
                    std::vector<u64> b(best, best + kLanes);
                    sort_list(b);
                    q.bound = std::max(q.bound, b[top - 1] - 1);
                }
            }
        }
        const bool all = (q.bound >> 32) == 0 || lanes > 8;
        const float low = value_of((unsigned)(q.bound >> 32));
        for (int lane = 0; lane < kLanes; lane++)
            for (int g = 0; g < kLpVals; g += 4) {
                const float four = fmaxf(fmaxf(v[lane][g], v[lane][g + 1]), fmaxf(v[lane][g + 2], v[lane][g + 3]));
                if (!all && !(four >= low)) continue;
                for (int e = g; e < g + 4; e++)
                    if ((all || v[lane][e] >= low) && key[lane][e] > q.bound) q.waiting.push_back(key[lane][e]);
            }
        most_waiting = std::max(most_waiting, (int)q.waiting.size());
        if (most_waiting > kLpWaiting) return false;
        while (q.waiting.size() >= kLanes) {
            q.list.insert(q.list.end(), q.waiting.end() - kLanes, q.waiting.end());
            q.waiting.resize(q.waiting.size() - kLanes);
            sort_list(q.list);
            q.list.resize(kLanes, 0);
            q.bound = std::max(q.bound, q.list[top - 1]);
        }
        if (q.bound > before) published.push_back(std::max(q.bound, published.back()));
        return true;
    }
};

}  // namespace

// Runs `count` orders of the waves' steps (the first few one wave after the
// other, last wave first among them; then by chance) over one row.  0: the ids
// are `want` in all of them; 1: wrong ids (the last ones in `got`); 2: more keys
// than the buffer holds.  most_waiting: the most that waited.
extern "C" int logprobs_orders(const float *l, int n, int skip, int vec, int top, int count, unsigned seed,
                               const int *want, int *got, int *most_waiting) {
    std::mt19937 rng(seed);
    const int steps = (n + skip + kStep - 1) / kStep;
    *most_waiting = 0;
    for (int o = 0; o < count; o++) {
        std::vector<int> order;
        for (int wave = 0; wave < kWaves; wave++) order.insert(order.end(), steps, o == 0 ? kWaves - 1 - wave : wave);
        if (o == 2) {
            for (int i = 0; i < kWaves * steps; i++) order[i] = kWaves - 1 - i % kWaves;
        } else if (o > 2) {
            std::shuffle(order.begin(), order.end(), rng);
        }
        Model m{l, n, skip, vec, top};
        int next[kWaves] = {};
        bool fits = true;
        for (size_t i = 0; i < order.size() && fits; i++) {
            const int wave = order[i];
            const int newest = (int)m.published.size() - 1;
            int &read = m.w[wave].read;
            read = o % 2 ? newest : std::max(read, newest - (int)(rng() % 4));
            fits = m.step(wave, next[wave]++, m.published[o < 3 ? newest : read]);
        }
        *most_waiting = std::max(*most_waiting, m.most_waiting);
        if (!fits) return 2;
        std::vector<u64> all;
        for (const Wave &q : m.w) {
            all.insert(all.end(), q.list.begin(), q.list.end());
            all.insert(all.end(), q.waiting.begin(), q.waiting.end());
        }
        std::sort(all.begin(), all.end(), std::greater<u64>());
        all.resize(std::max(all.size(), (size_t)top), 0);
        bool same = true;
        for (int i = 0; i < top; i++) {
            got[i] = (int)~(unsigned)all[i];
            same &= got[i] == want[i];
        }
        if (!same) return 1;
    }
    return 0;
}

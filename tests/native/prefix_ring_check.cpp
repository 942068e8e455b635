// The ring of the attention over a shared prefix, checked by itself on the host: the loaders, the
// two issuers and the softmax of a CTA as agents that run in any order, over barriers whose waits
// see only the parity of a phase. No unit may be put where the one before is still read, none read
// before it is there, nobody may wait forever, and whenever a CTA would have to give up, the units
// whose copies it waits for are all that may be on their way.
#define __host__
#define __device__
#include <cstdio>
#include <random>
#include <vector>

#include "prefix_plan.cuh"

using namespace skinny;

// Stages that keys and values take in turn: what the ring must not be for an odd number.
template <int kStages>
struct InTurn {
    static constexpr int kKeys = (kStages + 1) / 2, kValues = kStages / 2;
    static int stage(int unit) { return unit % kStages; }
    static int round(int unit) { return unit / kStages; }
    static int first_on_its_way(int end) { return end % 2; }
};

// As many units of a kind waited for as half the stages: one too few of the keys' for an odd number.
template <int kStages>
struct HalfDrained : PrefixRing<kStages> {
    static int first_on_its_way(int end) { return end - kStages / 2 * 2; }
};

struct Barrier {
    int phase = 0;
    bool complete(int parity) const { return (phase & 1) != parity; }  // the phase with this parity
    void arrive() { ++phase; }                                         // of one arrival each here
};

// 0, or what went wrong. `lag`: copies of a kind that are on their way before the oldest is
// published (0: each by itself, at any time).
template <class Ring, int kStages>
int simulate(unsigned seed, int steps, int lag) {
    std::mt19937 rng(seed);
    Barrier full[kStages], empty[kStages], scores, read, weights, product;
    int unit_at[kStages], state[kStages];  // 0 free, 1 being filled, 2 full
    for (int s = 0; s < kStages; ++s) unit_at[s] = -1, state[s] = 0;
    int next[2] = {0, 1}, landed[2] = {0, 1};        // loaders: unit to load, unit to publish
    int s_next = 0, s_done = 0, s_part = 0;          // products begun and complete (of which the first commit)
    int v_next = 0, v_done = 0, v_part = 0;
    int soft = 0, soft_part = 0;
    // How often each agent is let run, of 16: any of them may be slow for a while.
    int often[8];
    for (int n = 0, idle = 0; v_done < steps; ++n) {
        if (n % 64 == 0)
            for (int &o : often) o = rng() % 4 == 0 ? 1 : 1 + static_cast<int>(rng() % 16);
        const int who = static_cast<int>(rng() % 8);
        if (++idle > 40000) return 5;  // everybody waits
        if (static_cast<int>(rng() % 16) >= often[who]) continue;
        if (who < 2) {  // loader of keys, of values
            const int u = next[who], s = Ring::stage(u);
            if (u >= 2 * steps || !empty[s].complete((Ring::round(u) & 1) ^ 1)) continue;
            if (state[s] != 0) return 1;
            unit_at[s] = u, state[s] = 1, next[who] += 2;
            for (int t = 0; t < kStages; ++t)
                if (state[t] == 1 && unit_at[t] % 2 == who && unit_at[t] < Ring::first_on_its_way(next[who])) return 6;
        } else if (who < 4) {  // its copies land
            const int k = who - 2, u = landed[k], s = Ring::stage(u);
            const bool last = next[k] >= 2 * steps;
            if (u >= next[k] || (!last && next[k] - u <= 2 * lag)) continue;
            if (unit_at[s] != u || state[s] != 1) return 2;
            state[s] = 2, landed[k] += 2;
            full[s].arrive();
        } else if (who == 4) {  // the scores' issuer, and its products
            if (s_next < steps && s_next == s_done && (s_next == 0 || read.complete((s_next - 1) & 1)) &&
                full[Ring::stage(2 * s_next)].complete(Ring::round(2 * s_next) & 1)) {
                const int s = Ring::stage(2 * s_next);
                if (unit_at[s] != 2 * s_next || state[s] != 2) return 3;
                ++s_next;
            } else if (s_next > s_done && s_part == 0) {
                scores.arrive();
                s_part = 1;
            } else if (s_next > s_done) {
                const int s = Ring::stage(2 * s_done);
                if (unit_at[s] != 2 * s_done || state[s] != 2) return 3;
                state[s] = 0, s_part = 0, ++s_done;
                empty[s].arrive();
            } else {
                continue;
            }
        } else if (who == 5) {  // the output's issuer
            const int u = 2 * v_next + 1, s = Ring::stage(u);
            if (v_next >= steps || v_next != v_done || !full[s].complete(Ring::round(u) & 1) || !weights.complete(v_next & 1)) continue;
            if (unit_at[s] != u || state[s] != 2) return 4;
            ++v_next;
        } else if (who == 6) {  // its products
            if (v_next == v_done) continue;
            const int s = Ring::stage(2 * v_done + 1);
            if (unit_at[s] != 2 * v_done + 1 || state[s] != 2) return 4;
            if (v_part == 0) {
                product.arrive();
                v_part = 1;
            } else {
                state[s] = 0, v_part = 0, ++v_done;
                empty[s].arrive();
            }
        } else {  // the softmax
            if (soft >= steps) continue;
            if (soft_part == 0) {
                if (!scores.complete(soft & 1)) continue;
                read.arrive();
                soft_part = 1;
            } else {
                if (soft > 0 && !product.complete((soft - 1) & 1)) continue;
                weights.arrive();
                soft_part = 0, ++soft;
            }
        }
        idle = 0;
    }
    return 0;
}

template <int kStages>
bool check() {
    bool caught = kStages % 2 == 0, missed = caught;  // in turn they are apart anyway
    for (unsigned seed = 0; seed < 3000; ++seed)
        for (int lag = 0; lag < PrefixRing<kStages>::kValues; ++lag) {
            const int bad = simulate<PrefixRing<kStages>, kStages>(seed, 40, lag);
            if (bad) {
                std::printf("%d: stages %d seed %u lag %d\n", bad, kStages, seed, lag);
                return false;
            }
            caught = caught || simulate<InTurn<kStages>, kStages>(seed, 40, lag) != 0;
            missed = missed || simulate<HalfDrained<kStages>, kStages>(seed, 40, lag) == 6;
        }
    if (!caught || !missed) std::printf("stages %d: nothing found in turn, or half drained\n", kStages);
    return caught && missed;
}

int main() {
    if (!check<4>() || !check<5>() || !check<6>() || !check<7>() || !check<8>()) return 1;
    std::printf("ok\n");
    return 0;
}

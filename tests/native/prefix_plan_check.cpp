// The plan of the attention over a shared prefix, checked by itself on the host: every tile of
// every key head and block belongs to one CTA, the parts of different CTAs and key heads have
// slots of their own within the workspace, and the join finds them all.
#define __host__
#define __device__
#include <cstdio>
#include <vector>

#include "prefix_plan.cuh"

using namespace skinny;

static int check(int rows, int group, int kv_heads, int head_dim, int sms, long long length, int capacity, int own) {
    const PrefixPlan plan = prefix_plan(rows, group, head_dim);
    const int ctas = prefix_ctas(rows, kv_heads, head_dim, plan, capacity, own, sms);
    if (ctas < 1 || ctas > sms || (sms > 1 && ctas == sms && own < 100 && capacity < 100 && rows < 10)) return 7;
    const int lanes = prefix_lanes(plan.blocks, ctas);
    const long long tiles_of_table = (capacity + plan.tokens - 1ll) / plan.tokens * kv_heads;
    long long most = prefix_ranges(plan.blocks, ctas);
    if (most > tiles_of_table) most = tiles_of_table;
    if (most < 1 || most * lanes > ctas) return 1;
    const int steps = static_cast<int>((length + plan.tokens - 1) / plan.tokens);
    const PrefixCut cut(steps * kv_heads, static_cast<int>(most));
    const long long q = static_cast<long long>(rows) * group;
    const PrefixWorkspace ws = prefix_workspace(rows, group * kv_heads, kv_heads, head_dim, sms);
    const size_t slots = (ws.bytes - ws.slots) / (prefix_slot_floats(head_dim, q) * sizeof(float));
    std::vector<char> used(slots);
    int next = 0;
    for (int r = 0; r < cut.ranges; ++r) {
        if (cut.begin(r) != next || cut.begin(r + 1) <= next) return 2;
        next = cut.begin(r + 1);
        for (int x = cut.begin(r); x < next;) {
            const int head = x / steps, t = x - head * steps;
            const int n = steps - t < next - x ? steps - t : next - x;
            const int first = cut.owner(head * steps), last = cut.owner(head * steps + steps - 1);
            if (r < first || r > last || cut.owner(x) != r || cut.owner(x + n - 1) != r) return 3;
            for (int b = 0; b < plan.blocks; ++b) {
                const long long slot = static_cast<long long>(r + head) * plan.blocks + b;
                if (slot >= static_cast<long long>(slots) || used[slot]++) return 4;
            }
            x += n;
        }
    }
    if (next != steps * kv_heads) return 5;
    for (int head = 0; steps > 0 && head < kv_heads; ++head)
        for (int r = cut.owner(head * steps); r <= cut.owner(head * steps + steps - 1); ++r)
            if (!used[static_cast<size_t>(r + head) * plan.blocks]) return 6;
    return 0;
}

int main() {
    const int dims[] = {64, 96, 128, 192, 256}, all_rows[] = {1, 2, 17, 64, 130, 512, 1024}, groups[] = {1, 7, 16, 64, 128};
    const int all_kv[] = {1, 2, 7, 8}, all_sms[] = {1, 148, 152, 256}, lengths[] = {0, 1, 63, 64, 65, 509, 5001, 20011};
    for (int D : dims)
        for (int rows : all_rows)
            for (int group : groups)
                for (int kv : all_kv)
                    for (int sms : all_sms)
                        for (int length : lengths)
                            for (int capacity : {length > 0 ? length : 1, length + 16, 65536})
                                for (int own : {1, 1000})
                                    if (const int bad = check(rows, group, kv, D, sms, length, capacity, own)) {
                                        std::printf("%d: rows %d group %d kv %d D %d sms %d length %d capacity %d own %d\n", bad,
                                                    rows, group, kv, D, sms, length, capacity, own);
                                        return 1;
                                    }
    std::printf("ok\n");
    return 0;
}

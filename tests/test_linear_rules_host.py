"""The rules by which linear attention's plan cuts requests, compiled for the host."""
import os
import subprocess

from paged_variable_length_gb300 import build


def test_the_plan_cuts_only_where_the_host_launches_the_states_pass(tmp_path):
    """Whatever requests a batch holds, short ones and skipped ones (bad state slots) among them: where the plan cuts,
    the host launches the kernels that find the segments' states, and those fit the workspace.  Two batches by
    name: their skipped requests' tokens once told the plan, and not the host, that the others should be cut."""
    src = tmp_path / "rules.cpp"
    src.write_text(r'''
#include <cstdio>
#include <cstdlib>
#include "linear.h"
using namespace pva;
static int n[200], skipped[200];
static int check(int B, int hkv, int group, int sms, int hint) {
    long long total = 0, long_tokens = 0;
    int longest = 0;
    for (int i = 0; i < B; ++i) {
        total += n[i];
        if (n[i] <= kStepTokens) continue;
        long_tokens += n[i];
        if (n[i] > longest) longest = n[i];
    }
    const bool run = may_cut(total, B, hint > 0 && hint < total ? hint : (int)total, hkv, sms);
    // the plan's own rule never cuts where the host's bounds say no
    const int seg = segment_tokens(long_tokens, longest, hkv, sms);
    if (!run && seg != kWholeSegment) return printf("cut without a states pass: %d heads, %lld tokens\n", hkv, total), 1;
    // and whatever it were told of the tokens, it stays whole then
    long long fewer = 0;
    int least_longest = 0;
    for (int i = 0; i < B; ++i)
        if (n[i] > kStepTokens && !skipped[i]) fewer += n[i], least_longest = n[i] > least_longest ? n[i] : least_longest;
    if (!run && planned_segment_tokens(run, fewer, least_longest, hkv, sms) != kWholeSegment) return printf("planned\n"), 1;
    const int use = planned_segment_tokens(run, long_tokens, longest, hkv, sms);
    long long items = 0, with_state = 0;
    for (int i = 0; i < B; ++i) {
        if (n[i] <= kStepTokens || skipped[i]) continue;
        const int chunks = (n[i] + kChunk - 1) / kChunk, want = (int)(((long long)n[i] + use - 1) / use);
        const int per = (chunks + want - 1) / want, nseg = (chunks + per - 1) / per;
        items += nseg;
        if (nseg > 1) with_state += nseg;
    }
    if (head_parts(items, group, hkv, sms) > 1)
        for (int i = 0; i < B; ++i) with_state += n[i] > kStepTokens && !skipped[i] && n[i] <= use;
    if (with_state > 3 * (sms / hkv) + 3) return printf("%lld states, Hkv %d\n", with_state, hkv), 1;
    return 0;
}
int main() {
    for (int sms = 148; sms <= 160; sms += 4) {
        n[0] = 1024, n[1] = 1100, skipped[0] = 0, skipped[1] = 1;
        if (check(2, 32, 1, sms, 0)) return 1;
        for (int i = 0; i < 8; ++i) n[i] = 2000, skipped[i] = i > 0;
        if (check(8, 32, 1, sms, 0) || check(8, 32, 1, sms, 2000)) return 1;
        for (int i = 0; i < 3; ++i) n[i] = 1500, skipped[i] = i > 0;
        if (check(3, 32, 1, sms, 1500)) return 1;
    }
    srand(5);
    for (int round = 0; round < 40000; ++round) {
        const int B = 1 + rand() % (round % 2 ? 6 : 200);
        int longest = 0;
        for (int i = 0; i < B; ++i) {
            const int kind = rand() % 4;
            n[i] = kind == 0 ? rand() % (kStepTokens + 1) : kStepTokens + 1 + rand() % (kind == 1 ? 200 : kind == 2 ? 3000 : 30000);
            skipped[i] = rand() % 3 == 0;
            if (n[i] > longest) longest = n[i];
        }
        if (check(B, 1 + rand() % 40, 1 + rand() % 16, 152, round % 3 ? longest + rand() % 2 * 100 : 0)) return 1;
    }
    return 0;
}
''')
    exe = tmp_path / "rules"
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(build.CSRC), "-I", "/usr/local/cuda/include", str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout

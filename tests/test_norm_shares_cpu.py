"""How norm_rotary cuts its tokens: as many CTAs as it counts on fit an SM together, and no other share would end sooner by
its own measure."""
import random
import subprocess

SRC = r"""
#include <cstdio>
#include "norm_rotary.h"
using namespace kvevict;
// a line: tokens, heads, rows of a CTA at once, rotary_dim
int main()
{
    long long total, heads, step;
    int R;
    std::printf("%d %d %d %d\n", kNormCtas, kNormOwn, kNormPairs * 8, kNormStart);
    while (std::scanf("%lld %lld %lld %d", &total, &heads, &step, &R) == 4) std::printf("%d\n", norm_tokens(total, heads, step, R));
}
"""


def test_shares_fit_an_sm(tmp_path):
    (tmp_path / "s.cu").write_text(SRC)
    from kv_cache_eviction_decode_gb300 import build
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, str(tmp_path / "s.cu"), "-o", str(tmp_path / "s")],
                   check=True)
    r = random.Random(4)
    cases = [(32768, 72, 32, 128), (65536, 72, 32, 128), (131072, 72, 32, 128), (16384, 36, 16, 256), (16384, 72, 32, 128), (2**31 - 1, 131070, 8, 512)]
    for _ in range(300):
        lanes = r.choice([1, 2, 4, 8, 16, 32])
        cases.append((round(2 ** r.uniform(8, 24)), r.randint(1, 200), 256 // lanes, 2 * r.randint(0, lanes * 8)))
    out = subprocess.run([str(tmp_path / "s")], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True,
                         check=True).stdout.split("\n")
    ctas, own, static, start = map(int, out[0].split())
    assert ctas * 256 * 64 <= 65536  # threads and the launch bound's registers
    for (total, heads, step, R), line in zip(cases, out[1:]):
        t = int(line)

        def fits(n):
            return ctas * (own + static + n * (R // 2) * 8 + 1024) <= 228 * 1024

        def cost(n):
            return -(-(-(-total // n)) // (ctas * 152)) * (n * heads / step + start)
        assert 1 <= t <= 64 and fits(t), (total, heads, step, R, t)
        assert cost(t) <= 1.01 * min(cost(n) for n in range(1, 65) if fits(n)), (total, heads, step, R, t)

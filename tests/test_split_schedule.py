"""The split decode's distribution of work, from the kernel's own functions compiled for the host: whatever the
lengths, the window and the number of CTAs, every (sequence, KV head, block) triple belongs to exactly one CTA, and
the CTAs that share a group know each other and leave their parts in different places.  (CPU only.)"""
import os
import random
import subprocess
import tempfile
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent

PROBE = r"""
#include <cstdio>
#include <vector>
#include "decode_split.cuh"
using namespace pa;
int main()
{
    int B, h_kv, bs, ctas, window, max_blocks;
    while (std::scanf("%d %d %d %d %d %d", &B, &h_kv, &bs, &ctas, &window, &max_blocks) == 6) {
        std::vector<int> prefix(B + 1, 0), cuts(B + 1, 0);
        int longest = 0;
        for (int s = 0; s < B; ++s) {
            int ctx, first, n;
            if (std::scanf("%d", &ctx) != 1) return 1;
            split_blocks(ctx, window, bs, max_blocks, first, n);
            std::printf("seq %d %d\n", first, n);
            prefix[s + 1] = prefix[s] + n;
            longest = n > longest ? n : longest;
        }
        for (int s = 0; s < B; ++s) cuts[s + 1] = cuts[s] + ceil_div(prefix[s + 1] - prefix[s], split_piece(longest, bs));
        for (int c = 0; c < ctas; ++c) {
            const SplitRange r = split_range(prefix.data(), cuts.data(), B, h_kv, bs, longest, ctas, c);
            for (long long x = r.x0; x < r.x1;) {
                const SplitPlace at = split_locate(prefix.data(), B, h_kv, x);
                const long long left = r.x1 - x, n = at.nb - at.block < left ? at.nb - at.block : left, group0 = x - at.block;
                int c0, pieces;
                split_sharers(r, group0, at.nb, c0, pieces);
                std::printf("part %d %d %d %d %d %d %d %d %d %d\n", c, at.seq, at.kvh, at.block, (int)n, at.nb, c0, pieces,
                            split_slot(r, group0, c), (int)r.aligned);
                x += n;
            }
        }
        std::printf("end\n");
    }
}
"""


def _cases():
    rnd = random.Random(7)
    out = [(1, 1, 16, 444, 0, 10000, [131072]), (1, 8, 16, 148, 0, 100, [1001]), (3, 2, 32, 36, 0, 20, [0, 0, 0]),
           (2, 2, 16, 12, 64, 6, [37, 81]), (4, 1, 16, 3, 0, 4, [100, 2 ** 31 - 1, -5, 64]), (2, 4, 64, 1, 0, 99, [6000, 1])]
    for _ in range(300):
        B = rnd.choice([1, 2, 3, 7, 40, 300])
        top = rnd.choice([1, 20, 300, 513, 5000, 60000 if B < 8 else 2000])
        bs = rnd.choice([16, 32, 64])
        window = rnd.choice([0, 0, 1, 50, 1000])
        out.append((B, rnd.choice([1, 2, 5, 8]), bs, rnd.choice([1, 2, 17, 148, 444, 592, 1024]), window,
                    -(-top // bs) + rnd.choice([0, 3, -2 if top > 4 * bs else 0]), [rnd.randint(0, top) for _ in range(B)]))
    return out


@pytest.fixture(scope="module")
def answers():
    with tempfile.TemporaryDirectory() as tmp:
        src, exe = Path(tmp) / "probe.cu", Path(tmp) / "probe"
        src.write_text(PROBE)
        nvcc = "/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else "nvcc"
        subprocess.run([nvcc, "-std=c++17", "--expt-relaxed-constexpr", "-gencode", "arch=compute_100a,code=sm_100a",
                        "-I", str(ROOT / "include"), "-I", str(ROOT / "paged_kv_cache_428_b200" / "csrc"), str(src),
                        "-o", str(exe)], check=True, capture_output=True)
        cases = _cases()
        text = "".join(" ".join(map(str, (*c[:6], *c[6]))) + "\n" for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
    got, cur = [], []
    for line in out.splitlines():
        if line == "end":
            got.append(cur)
            cur = []
        else:
            f = line.split()
            cur.append((f[0], *map(int, f[1:])))
    assert len(got) == len(cases)
    return list(zip(cases, got))


def test_every_triple_once_and_sharers_agree(answers):
    aligned_seen = set()
    for (B, h_kv, bs, ctas, window, max_blocks, lens), lines in answers:
        seqs = [x[1:] for x in lines if x[0] == "seq"]
        for ctx, (first, n) in zip(lens, seqs):
            have = -(-max(ctx, 0) // bs)
            lo = (ctx - window) // bs if window and ctx > window else 0
            assert first == lo and n == (max(min(have, max(max_blocks, lo) + 1) - lo, 0) if ctx > 0 else 0)
        groups, per_cta = {}, {}
        for _, c, s, k, b, n, nb, c0, pieces, slot, aligned in (x for x in lines if x[0] == "part"):
            assert nb == seqs[s][1] and 0 <= k < h_kv and n > 0
            groups.setdefault((s, k), []).append((b, n, c, c0, pieces, slot))
            per_cta[c] = per_cta.get(c, 0) + n
            aligned_seen.add(aligned)
        assert set(groups) == {(s, k) for s in range(B) for k in range(h_kv) if seqs[s][1]}
        used = set()
        for (s, k), parts in groups.items():
            at = 0
            for i, (b, n, c, c0, pieces, slot) in enumerate(sorted(parts)):
                assert b == at and c == c0 + i and pieces == len(parts)       # in order, one a CTA, counted right
                at += n
                if len(parts) > 1:
                    assert 2 * c <= slot <= 2 * c + 1 and slot not in used    # a place of its own
                    used.add(slot)
            assert at == seqs[s][1] and len(parts) <= 64
        if per_cta and ctas > 1:                                              # nobody has much more than his share
            total, longest = sum(per_cta.values()), max(n for _, n in seqs)
            fair = max(-(-total // ctas), 128 // bs, -(-longest // 62), longest if longest * bs <= 512 else 0)
            assert max(per_cta.values()) <= fair
    assert aligned_seen == {0, 1}

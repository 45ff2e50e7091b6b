"""Which attention kernel a call takes, and how the prompt kernel's groups are cut, without a GPU: both are worked out on the host."""
import subprocess

import pytest

from plan_testlib import ask, compiled

SOURCE = r"""
#include "attn_plan.h"
#include <cmath>
#include <cstdio>
#include <initializer_list>
using namespace moe::attn;

// The prompt kernel's tiles of one group of 256 rows, as it finds them on the device.
static long long tiles(const Call& c, long long n, long long len, long long rt)
{
    const long long rows = n * c.group - rt * 256 < 256 ? n * c.group - rt * 256 : 256;
    const long long pos0 = len - n + rt * 256 / c.group, pos1 = len - n + (rt * 256 + rows - 1) / c.group;
    const long long first = c.window > 0 && pos0 >= c.window ? (pos0 - c.window + 1) / 128 : 0;
    return pos1 / 128 - first + 1;
}

static int fail(const Call& c, const char* what)
{
    std::printf("%s: %d sequences, %d tokens, group %d, %d heads of %d, block %d, format %d, stride %d, window %d\n", what, c.n_seqs,
                c.n_tokens, c.group, c.H, c.D, c.blk, c.fmt, c.table_stride, c.window);
    return 1;
}

static int sweep()
{
    const int groups[] = {1, 3, 8, 16, 80}, windows[] = {0, 1, 128, 700, 1 << 30}, tokens[] = {1, 2, 7, 63, 300, 5000}, formats[] = {1, 2, 4};
    long long cuts = 0;
    for (int seqs : {1, 2, 5, 39, 1024})
        for (int each : tokens)
            for (int group : groups)
                for (int H : {1, 8, 19})
                    for (int window : windows)
                        for (int stride : {1, 10, 63, 70000})
                            for (int fmt : formats) {
                                const Call c{seqs, seqs * each < 1 << 20 ? seqs * each : 1 << 20, group, H, fmt == 2 ? 128 : 64, 64, fmt, stride, window};
                                const moe::PromptCut cut = prompt_cut(c, 152);
                                const long long most = ((long long)c.n_tokens * group + 255ll * (seqs < c.n_tokens ? seqs : c.n_tokens)) / 256 * H;
                                if (cut.whole + (long long)cut.rest != most)
                                    return fail(c, "groups are missing");
                                if (cut.rest && (cut.parts < 2 || cut.parts * cut.rest > 152 || cut.whole % 152 || cut.parts * 4 > pieces(c, 256, 128)))
                                    return fail(c, "a cut that cannot be");
                                if (!cut.rest && cut.parts != 1)
                                    return fail(c, "parts of nothing");
                                const double a = decode_ns(c, 152), b = prompt_ns(c, 152);
                                if (!(a > 0) || !(b > 0) || !std::isfinite(a) || !std::isfinite(b))
                                    return fail(c, "no time");
                                cuts += cut.rest > 0;
                                // no group has more tiles than `pieces` says
                                const long long held = (long long)stride * 64;
                                for (long long len : {(long long)each, held / 3, held / 2 + 17, held - 1, held})
                                    if (len >= each && len <= held)
                                        for (long long rt = 0; rt * 256 < (long long)each * group; rt += 1 + rt / 3)
                                            if (tiles(c, each, len, rt) > pieces(c, 256, 128))
                                                return fail(c, "a group sees more");
                            }
    std::printf("%lld\n", cuts);
    return cuts > 100 ? 0 : 1;
}

int main() { return sweep(); }
"""

# Measured: us of the decode / prompt kernel, for 1 and then 8 sequences of 1, 6, 8 and 16 tokens.  The columns before:
# format, head size, query heads, kv heads, keys, window (0: none).
MEASURED = """
    1 64 64 8 4000 128  7.1/10.7 8.0/10.7 8.6/10.9 9.7/11.9 7.4/10.9 12.2/11.0 13.2/11.1 15.2/12.1
    1 64 64 8 600 0  9.8/12.6 10.9/13.0 14.8/13.0 16.0/14.1 14.6/12.9 20.9/13.2 22.6/13.4 29.2/14.3
    1 64 64 8 4000 0  15.2/14.8 18.7/15.0 19.9/15.2 23.4/16.2 22.0/28.2 37.9/28.7 44.9/28.9 75.5/44.7
    1 64 64 8 16000 0  18.9/22.6 25.6/24.2 29.4/24.4 44.2/25.7 43.2/81.1 100.1/82.6 127.8/82.6 241.1/150.8
    1 128 32 4 4000 128  7.9/12.5 9.9/13.2 10.2/13.6 11.5/15.6 8.4/12.8 10.3/13.4 10.7/13.6 18.2/16.0
    1 128 32 4 600 0  11.3/15.5 14.0/16.0 14.2/16.5 18.9/18.8 14.6/15.6 24.2/16.2 24.8/16.7 30.4/18.7
    1 128 32 4 4000 0  18.9/17.5 22.0/18.3 24.9/18.5 26.6/20.6 21.9/22.9 33.5/24.1 38.8/24.5 59.1/31.0
    1 128 32 4 16000 0  22.4/27.4 27.4/29.2 32.1/29.7 39.1/31.6 35.5/54.0 74.1/57.0 90.7/57.5 162.3/73.1
    4 64 64 8 4000 128  7.3/11.5 8.4/11.8 8.6/11.7 9.9/12.5 7.6/12.1 10.8/12.1 10.9/12.2 17.4/12.6
    4 64 64 8 600 0  9.2/13.8 10.1/14.0 10.5/14.1 11.7/14.4 9.4/14.0 15.2/14.2 15.6/14.4 24.5/14.8
    4 64 64 8 4000 0  16.2/15.8 19.7/15.9 20.6/16.0 24.0/16.4 21.8/31.0 37.5/31.2 44.0/31.3 73.3/49.3
    4 64 64 8 16000 0  19.0/23.7 26.6/25.5 29.9/25.7 43.1/26.7 34.1/89.4 95.9/91.6 122.9/91.4 230.1/172.2
    4 128 32 4 4000 128  8.2/13.1 11.0/13.6 11.2/13.6 12.3/15.7 8.6/13.2 11.7/13.7 11.8/13.9 16.3/15.6
    4 128 32 4 600 0  11.1/15.6 14.0/16.2 14.3/16.5 15.4/18.1 11.7/15.8 14.6/16.4 14.8/16.8 23.8/18.1
    4 128 32 4 4000 0  19.5/17.6 24.3/18.1 23.9/18.6 30.3/19.9 22.9/23.4 37.8/24.4 42.7/24.9 64.4/31.1
    4 128 32 4 16000 0  21.6/27.2 32.2/29.2 35.2/29.6 42.7/31.0 31.8/56.9 80.2/59.4 99.3/59.7 177.6/77.6
"""


def ask64(calls):
    """For calls (sequences, tokens of each, query heads, kv heads, head size, format, keys that the table holds, window), in blocks of 64."""
    return ask([(b, b * n, hq, h, d, 64, f, -(-keys // 64), w) for b, n, hq, h, d, f, keys, w in calls])


def test_every_call_is_cut_soundly(tmp_path):
    r = subprocess.run([compiled(SOURCE, str(tmp_path))], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_faster_kernel():
    """Against both kernels' measured times: never much behind the better one, and hardly ever by more than a tenth."""
    calls, times = [], []
    for line in MEASURED.strip().splitlines():
        f, d, hq, h, keys, w, *pairs = line.split()
        for (b, n), pair in zip([(b, n) for b in (1, 8) for n in (1, 6, 8, 16)], pairs):
            calls.append((b, n, int(hq), int(h), int(d), int(f), int(keys), int(w)))
            times.append(tuple(map(float, pair.split("/"))))
    loss = [t[took] / min(t) for (took, _), t in zip(ask64(calls), times)]
    assert len(loss) == 128 and max(loss) <= 1.25
    assert sum(x > 1.1 for x in loss) <= 10
    assert sum(loss) / len(loss) <= 1.02


@pytest.mark.parametrize("fmt", [1, 2, 4])
@pytest.mark.parametrize("hq,h,d", [(64, 8, 64), (32, 4, 128)])
def test_few_tokens_within_a_window_or_of_short_sequences(fmt, hq, h, d):
    """A handful of tiles gets no parts: the decode kernel, whose work lies over all SMs, however wide the table is."""
    calls = [(b, n, hq, h, d, fmt, keys, 128) for b in (1, 2, 4) for n in (1, 4, 5, 6, 7, 8) for keys in (300, 4000, 1 << 17)]
    calls += [(b, n, hq, h, d, fmt, 300, 0) for b in (1, 2, 4) for n in (1, 4, 5, 6, 7, 8)]
    assert all(answer == (0, 1) for answer in ask64(calls))


@pytest.mark.parametrize("fmt", [1, 2, 4])
def test_many_rows_over_many_keys(fmt):
    """The prompt kernel, in parts where its groups are few."""
    few, many = ask64([(1, 16, 64, 8, 64, fmt, 16000, 0), (2, 2100, 32, 4, 128, fmt, 5100, 0)])
    assert few == (1, 19) and many[0] == 1


def test_single_tokens_of_long_sequences():
    calls = [(b, 1, hq, h, d, f, keys, 0) for f in (1, 2, 4) for hq, h, d in ((64, 8, 64), (32, 4, 128)) for b in (1, 4, 64) for keys in (8000, 16000, 1 << 17)]
    assert all(took == 0 for took, _ in ask64(calls))

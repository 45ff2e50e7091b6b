"""The host's choice between the attention kernels (csrc/attn_plan.h), for tests that are about one of them."""
from __future__ import annotations

import os
import subprocess
import tempfile

from bit_moe_decode_02_gb300 import build_ext

SOURCE = r"""
#include "attn_plan.h"
#include <cstdio>
int main()
{
    moe::attn::Call c;
    while (std::scanf("%d %d %d %d %d %d %d %d %d", &c.n_seqs, &c.n_tokens, &c.group, &c.H, &c.D, &c.blk, &c.fmt, &c.table_stride, &c.window) == 9)
        std::printf("%d %d\n", (int)moe::attn::takes_prompt_kernel(c, 152), moe::attn::prompt_cut(c, 152).parts);
    return 0;
}
"""
_exe = None


def compiled(source, where):
    src, exe = os.path.join(where, "plan.cpp"), os.path.join(where, "plan")
    with open(src, "w") as f:
        f.write(source)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", build_ext.CSRC, "-I", os.path.join(build_ext.ROOT, "include"), src, "-o", exe],
                   check=True)
    return exe


def ask(calls):
    """For calls (sequences, tokens in all, query heads, kv heads, head size, block, format, table's width, window): whether the prompt
    kernel takes it on 152 SMs, and the most parts that it cuts a group's keys into."""
    global _exe
    if _exe is None:
        _exe = compiled(SOURCE, tempfile.mkdtemp())
    text = "".join(f"{s} {t} {hq // h} {h} {d} {blk} {f} {st} {w}\n" for s, t, hq, h, d, blk, f, st, w in calls)
    r = subprocess.run([_exe], input=text, capture_output=True, text=True, check=True)
    return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]


def in_parts(c, new, heads, window=0) -> bool:
    """Whether a call over the cache c (ops_testlib) takes the prompt kernel with some keys in parts."""
    (took, parts), = ask([(len(new), sum(new), heads, c.H, c.D, c.blk, c.fmt, c.dtable.shape[1], window)])
    return took == 1 and parts > 1

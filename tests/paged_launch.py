"""The launches that the paged attention's rule on sizes chooses: lf_paged.h's plan_attn, compiled for the host."""
import os
import subprocess
from collections import namedtuple

from conftest import ROOT

Launch = namedtuple("Launch", "cl cw parts sorted")

SOURCE = """
#include <cstdio>
#include "persistent_monokernel_gb300/csrc/lf_paged.h"
int main()
{
    lfpg::Attn a = {};
    int sms;
    while (std::scanf("%d %d %d %d %d %d %d %d", &a.n, &a.G, &a.c.Hkv, &a.c.hd, &a.c.page, &a.width, &a.win, &sms) == 8) {
        lfpg::plan_attn(a, sms);
        std::printf("%d %d %d %d\\n", a.cl, a.cw, a.parts, a.sorted);
    }
}
"""


def launches(queries, folder, sms=152):
    """[Launch] of queries (rows, heads per KV head, KV heads, head_dim, page, columns of the table, window)."""
    from persistent_monokernel_gb300 import build
    src, exe = os.path.join(folder, "launch.cpp"), os.path.join(folder, "launch")
    with open(src, "w") as f:
        f.write(SOURCE)
    include = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-I", ROOT, "-I", include, src, "-o", exe], check=True)
    text = "\n".join(" ".join(map(str, (*q, sms))) for q in queries)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
    return [Launch(*map(int, line.split())) for line in out.splitlines()]

"""The block-scaled e4m3 tiles count the loads behind their copies: at the barrier of two groups they wait until at most N
vector loads are in flight, which says that the groups' copies have landed in LDS only if N loads or more were issued after
them; and the copies of the next two groups may go to their stages only behind that barrier.  Both are orders that the
compiler has to keep, under every scheduling strategy, not only the default one: the device code is built under several and
its loads are counted."""
import os
import re
import subprocess

import pytest

from rank_error_compensation_amd import build as B

STRATEGIES = ["default", "gcn-max-ilp", "gcn-iterative-ilp", "gcn-iterative-minreg", "gcn-max-memory-clause"]


def assembly(strategy, path):
    cmd = [B.hipcc(), "-x", "hip", "--offload-device-only", "-S", os.path.join(B.CSRC, "fp8.hip"), "-o", str(path)]
    cmd += B.common_flags()
    if strategy != "default":
        cmd += ["-mllvm", f"-misched={strategy}"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0 and "Cannot find option" in p.stderr:
        pytest.skip(f"this compiler has no strategy {strategy}")
    assert p.returncode == 0, p.stderr[-2000:]
    return path.read_text()


def kernels(text):
    """(template arguments, events) of every tile kernel: ("copy"), ("load"), ("wait", n), ("barrier")."""
    for m in re.finditer(r"^(_ZN\S*fp8_tile_kernelI((?:L[ib]\d+E)+)\S*):.*?\n(.*?)^\.Lfunc_end", text, re.M | re.S):
        args = [int(v) for v in re.findall(r"L[ib](\d+)E", m.group(2))]
        events = []
        for line in m.group(3).split("\n"):
            t = line.strip()
            if t.startswith("global_load_lds_dwordx4"):
                events.append(("copy",))
            elif re.match(r"(global|flat|buffer)_load", t):
                events.append(("load",))
            elif t.startswith("s_waitcnt") and "vmcnt" in t:
                events.append(("wait", int(re.search(r"vmcnt\((\d+)\)", t).group(1))))
            elif t.startswith("s_barrier"):
                events.append(("barrier",))
        yield args, events


def check(args, events):
    """Preamble and three turns of the loop, in the order of the code."""
    wm, wn, tt = args[:3]
    per = 2 * (16 * tt * wm // 8 // (wm * wn)) + 1  # copies of two groups per wavefront, and their scales
    at = [i for i, e in enumerate(events) if e[0] == "barrier" and events[i - 1][0] == "wait" and events[i - 1][1] > 0]
    assert len(at) == 2, (args, len(at))  # a turn of four stages, two at a barrier
    end = next(i for i in range(at[-1] + 1, len(events)) if events[i][0] == "barrier")
    body = events[at[0] - 1:end - 1]
    start = next(i for i, e in enumerate(events) if e[0] == "copy")
    copies, behind, allowed, seen = 0, 0, None, 0
    for e in events[start:at[0] - 1] + 3 * body:
        if e[0] == "copy":
            copies, behind = copies + 1, 0
        elif e[0] == "load":
            behind += 1
        elif e[0] == "wait":
            allowed = e[1]
        else:
            assert copies == per, f"tile {args}: {copies} copies in front of barrier {seen}, two groups have {per}"
            assert behind >= allowed, f"tile {args}: {behind} loads behind the copies of barrier {seen}, its wait allows {allowed} in flight"
            copies, seen = 0, seen + 1
    assert seen == 6


@pytest.mark.parametrize("strategy", STRATEGIES)
def test_copies_have_landed_at_their_barrier(strategy, tmp_path):
    found = list(kernels(assembly(strategy, tmp_path / "fp8.s")))
    assert len(found) >= 9
    for args, events in found:
        check(args, events)

"""The 8-bit integer tiles count the loads behind a copy: at the barrier of a group they wait until at most N
vector loads are in flight, which says that the group's copies have landed in LDS only if N loads or more were
issued after them.  That is an order the compiler has to keep, under every scheduling strategy, not only the
default one: the device code is built under several and its loads are counted."""
import os
import re
import subprocess

import pytest

from rank_error_compensation_amd import build as B

STRATEGIES = ["default", "gcn-max-ilp", "gcn-iterative-ilp", "gcn-iterative-minreg", "gcn-max-memory-clause"]


def assembly(strategy, path):
    cmd = [B.hipcc(), "-x", "hip", "--offload-device-only", "-S", os.path.join(B.CSRC, "w8a8.hip"), "-o", str(path)]
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
    for m in re.finditer(r"^(_ZN\S*w8a8_tile_kernelI((?:Li\d+E)+)\S*):.*?\n(.*?)^\.Lfunc_end", text, re.M | re.S):
        args = [int(v) for v in re.findall(r"Li(\d+)E", m.group(2))]
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
    """Preamble and three turns of the ring, in the order of the code: the loads issued after a group's last
    copy, at the group's barrier, against the wait in front of it."""
    wm, wn, tt = args[:3]
    per = 16 * tt * wm // 8 // (wm * wn)  # copies of a group per wavefront
    at = [i for i, e in enumerate(events) if e[0] == "barrier" and events[i - 1][0] == "wait" and events[i - 1][1] > 0]
    assert len(at) == 4, (args, len(at))  # one turn of four stages
    end = next(i for i in range(at[-1] + 1, len(events)) if events[i][0] == "barrier")
    body = events[at[0] - 1:end - 1]
    start = next(i for i, e in enumerate(events) if e[0] == "copy")
    issued, last, copies, group = 0, {}, 0, 0
    for e in events[start:at[0] - 1] + 3 * body:
        if e[0] in ("copy", "load"):
            issued += 1
            if e[0] == "copy":
                last[copies // per] = issued
                copies += 1
        elif e[0] == "wait":
            allowed = e[1]
        else:
            behind = issued - last[group]
            assert copies >= (group + 1) * per and behind >= allowed, \
                f"tile {args}: group {group} has {behind} loads behind its copies, the wait allows {allowed} in flight"
            group += 1
    assert group == 12


@pytest.mark.parametrize("strategy", STRATEGIES)
def test_copies_have_landed_at_their_barrier(strategy, tmp_path):
    found = list(kernels(assembly(strategy, tmp_path / "w8a8.s")))
    assert len(found) >= 6
    for args, events in found:
        check(args, events)

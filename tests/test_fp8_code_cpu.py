"""What the block-scaled e4m3 tiles are compiled to.  A tile whose registers do not suffice moves some of them to scratch memory,
through the counter that the ring's waits count on; and of the tiles that correct, only the one of four teams reads the
projection as fp32 K ranges, so that only that one holds the code."""
import re

from test_fp8_schedule_cpu import assembly


def tiles(text):
    """(template arguments, instructions) of every tile kernel."""
    for m in re.finditer(r"^(_ZN\S*fp8_tile_kernelI((?:L[ib]\d+E)+)\S*):.*?\n(.*?)^\.Lfunc_end", text, re.M | re.S):
        lines = [line.strip() for line in m.group(3).split("\n") if line.startswith("\t")]
        yield [int(v) for v in re.findall(r"L[ib](\d+)E", m.group(2))], [t for t in lines if not t.startswith((".", ";"))]


def test_tiles_hold_their_registers_and_only_their_own_code(tmp_path):
    found = list(tiles(assembly("default", tmp_path / "fp8.s")))
    assert len(found) >= 9
    for args, code in found:
        wm, wn, tt, kh, mode, experts = args
        assert not [t for t in code if t.startswith("scratch_")], (args, "scratch")
        # roundings to fp16, two an instruction: the results alone (of a split launch the projection's join alone), and the
        # K ranges' sums of the projection in the correcting tile of several teams
        rounded = sum(t.startswith(("v_cvt_f16_f32", "v_cvt_pk_f16_f32")) for t in code)
        own = tt // kh * 4 * 4 // 2 if mode != 2 else 2
        print(args, len(code), rounded, own)
        assert rounded <= own or (mode == 1 and kh > 1), (args, rounded, own)
